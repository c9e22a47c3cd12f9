// gdr_tree: the gated delta rule for a tree of drafted tokens over a cached state.
//
// Node i of a tree has the state that the recurrence reaches over the nodes on
// its path; node j is on it if j is an ancestor of i.  With G_i the sum of g over
// the path to i, and D_ij = e^(G_i - G_j) for ancestors j of i, the corrected
// values and the outputs are those of the chunked form with the tree's mask:
//     (I + A) U = beta (V - e^G K h),     A_ij = beta_i D_ij (k_i . k_j), j an ancestor of i
//     O = scale (e^G Q h + P U),          P_ij = D_ij (q_i . k_j), j an ancestor of i, or i
// Parents come before their children, so A is strictly lower triangular.
//
// One workgroup per (sequence, v head), one wave per 32 value columns, nodes in
// NT tiles of 16.  The state is read once, straight into the registers that feed
// the products: lane (c, g) = (l & 15, l >> 4) of a wave loads h[32 kb + 8 g + i][2 c
// + t], the B operands of two 16-column tiles whose columns are 2 c and 2 c + 1.
// K, Q, A and P go through LDS.  The loads of the state are issued first and are in
// flight while the waves share out the 16 x 16 tiles of A and P and the inverses of
// I + A's diagonal tiles; after that each wave solves its own columns, tile by
// tile, with U in registers as the B operand of the next product.
//
// Non-finite values.  Node j must not reach nodes that are no descendants of it,
// though a product with a masked zero would turn its NaN or infinity into NaN there.
// Products by rows keep to their rows; entries of A and right-hand sides that are
// not finite are replaced by zero and remembered (by node, or by node and column),
// and the rows of those nodes and of their descendants are written as NaN.
#include "gdr_lds.hpp"
#include "gdr_pool.hpp"

namespace gdr {
namespace {

constexpr int LDT = 20;  // floats per row of a 16 x 16 tile in LDS (16 and padding: conflict-free rows)

template <typename In, int K, int NT> struct TreeLds {
    static constexpr int ROWB = K * sizeof(In) + 16;  // a row of K or Q with padding
    static constexpr int TILES = NT * (NT + 1) / 2;
    static constexpr int k = 0, q = k + 16 * NT * ROWB, a = q + 16 * NT * ROWB, p = a + TILES * 16 * LDT * 4,
                         G = p + TILES * 16 * LDT * 4, mask = G + 16 * NT * 8, eg = mask + 16 * NT * 8,
                         beta = eg + 16 * NT * 4, bad = beta + 16 * NT * 4, bytes = bad + 16;
};

__device__ __forceinline__ bool finite(float x) { return fabsf(x) < __builtin_inff(); }
// tile (r, c) of a lower triangle of 16 x 16 tiles
__device__ __forceinline__ int tile_at(int r, int c) { return (r * (r + 1) / 2 + c) * 16 * LDT; }

// fp32 product of a 16 x 16 tile of LDS (A operand) and an accumulator tile
__device__ __forceinline__ f32x4 tile_mul(const float *tile, f32x4 b, f32x4 c) {
    const f32x4 a = *reinterpret_cast<const f32x4 *>(tile + ln16() * LDT + 4 * lg4());
#pragma unroll
    for (int j = 0; j < 4; ++j) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[j], b[j], c, 0, 0, 0);
    return c;
}

// eight consecutive values of an operand's row, and a tile's product over 32 of them
template <typename In> struct Row8;
template <> struct Row8<bf16> {
    bf16x8 x;
    __device__ __forceinline__ void load(const char *p) { x = *reinterpret_cast<const bf16x8 *>(p); }
    __device__ __forceinline__ f32x4 dot(const Row8 &b, f32x4 c) const {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(x, b.x, c, 0, 0, 0);
    }
};
template <> struct Row8<float> {
    f32x4 x0, x1;
    __device__ __forceinline__ void load(const char *p) {
        x0 = *reinterpret_cast<const f32x4 *>(p);
        x1 = *reinterpret_cast<const f32x4 *>(p + 16);
    }
    __device__ __forceinline__ f32x4 dot(const Row8 &b, f32x4 c) const {
#pragma unroll
        for (int j = 0; j < 4; ++j) c = __builtin_amdgcn_mfma_f32_16x16x4f32(x0[j], b.x0[j], c, 0, 0, 0);
#pragma unroll
        for (int j = 0; j < 4; ++j) c = __builtin_amdgcn_mfma_f32_16x16x4f32(x1[j], b.x1[j], c, 0, 0, 0);
        return c;
    }
};

// eight state values of a column as an operand.  With bf16 rows the state is the sum
// of PIECES bf16 values: 3 keep 24 bits (an fp32 output), 2 keep 16 (a bf16 output has 8).
template <typename In, int PIECES> struct State8;
template <int PIECES> struct State8<bf16, PIECES> {
    bf16x8 x[PIECES];
    __device__ __forceinline__ void set(const float *h) {
        float r[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) r[i] = h[i];
#pragma unroll
        for (int s = 0; s < PIECES; ++s)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                x[s][i] = (bf16)r[i];
                r[i] -= (float)x[s][i];
            }
    }
    __device__ __forceinline__ f32x4 dot(const Row8<bf16> &a, f32x4 c) const {
#pragma unroll
        for (int s = PIECES - 1; s >= 0; --s) c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.x, x[s], c, 0, 0, 0);
        return c;
    }
};
template <int PIECES> struct State8<float, PIECES> {
    Row8<float> x;
    __device__ __forceinline__ void set(const float *h) {
        x.x0 = f32x4{h[0], h[1], h[2], h[3]};
        x.x1 = f32x4{h[4], h[5], h[6], h[7]};
    }
    __device__ __forceinline__ f32x4 dot(const Row8<float> &a, f32x4 c) const { return a.dot(x, c); }
};

typedef float pair __attribute__((ext_vector_type(2)));
__device__ __forceinline__ pair load2(const float *p) { return *reinterpret_cast<const pair *>(p); }
__device__ __forceinline__ pair load2(const bf16 *p) {
    return __builtin_convertvector(*reinterpret_cast<const bf16x2 *>(p), pair);
}
__device__ __forceinline__ void store2(float *p, pair x) { *reinterpret_cast<pair *>(p) = x; }
__device__ __forceinline__ void store2(bf16 *p, pair x) {
    *reinterpret_cast<bf16x2 *>(p) = __builtin_convertvector(x, bf16x2);
}

template <typename In, typename Out, int K, int V, int NT>
__global__ __launch_bounds__(2 * V, 2) void gdr_tree_kernel(PoolParams p) {
    using L = TreeLds<In, K, NT>;
    constexpr int NTHREADS = 2 * V, NW = V / 32, PIECES = sizeof(Out) == 4 ? 3 : 2;
    extern __shared__ __align__(16) char smem[];
    float *At = reinterpret_cast<float *>(smem + L::a), *Pt = reinterpret_cast<float *>(smem + L::p);
    double *G = reinterpret_cast<double *>(smem + L::G);
    uint64_t *mask = reinterpret_cast<uint64_t *>(smem + L::mask);
    float *eg = reinterpret_cast<float *>(smem + L::eg), *beta = reinterpret_cast<float *>(smem + L::beta);
    unsigned *bad = reinterpret_cast<unsigned *>(smem + L::bad);  // two words of node bits

    const int unit = blockIdx.x, j = unit / p.Hv, hv = unit - j * p.Hv, hq = hv / (p.Hv / p.Hq);
    const int l = lane_id(), w = __builtin_amdgcn_readfirstlane(wave_id()), c = ln16(), g = lg4();
    const int col = 32 * w + 2 * c;
    int64_t bos, eos;
    token_range(p, j, bos, eos);
    if (bos >= eos) return;
    const int slot = slot_of(p, j);
    Out *o = reinterpret_cast<Out *>(p.o) + hv * V;
    if (slot < 0 || eos - bos > TREE_MAX) {
        const float fill = slot < 0 ? 0.f : __builtin_nanf("");
        for (int64_t i = bos * V + threadIdx.x; i < eos * V; i += NTHREADS) o[i / V * p.Hv * V + i % V] = (Out)fill;
        return;
    }
    const int n = (int)(eos - bos), nt = (n + 15) >> 4;

    // K and Q, zero past the last node, to LDS
    constexpr int PER = Vec16<In>::n, CHUNKS = K / PER, TURNS = (16 * NT * CHUNKS + NTHREADS - 1) / NTHREADS;
    typedef typename Vec16<In>::type V16;
    V16 kx[TURNS], qx[TURNS];
    {
        const In *kp = reinterpret_cast<const In *>(p.k) + hq * K, *qp = reinterpret_cast<const In *>(p.q) + hq * K;
#pragma unroll
        for (int t = 0; t < TURNS; ++t) {
            const int at = t * NTHREADS + threadIdx.x, i = at / CHUNKS, d = at % CHUNKS * PER;
            kx[t] = V16{};
            qx[t] = V16{};
            if (i < n) {
                kx[t] = *reinterpret_cast<const V16 *>(kp + row_offset(p, j, bos + i, p.k_batch, p.k_row) + d);
                qx[t] = *reinterpret_cast<const V16 *>(qp + row_offset(p, j, bos + i, p.q_batch, p.q_row) + d);
            }
        }
    }
    // wave 0: parents, gates and beta, a node per lane
    int up = -1;
    float gate = 0.f, b = 0.f;
    if (w == 0 && l < n) {
        up = p.parents[bos + l];
        gate = p.g[(bos + l) * p.Hv + hv];
        b = p.beta[(bos + l) * p.Hv + hv];
    }
    // the state
    pair h[K / 32][8];
    {
        const float *hp = p.states + (int64_t)slot * p.slot_stride + ((int64_t)hv * K + 8 * g) * V + col;
#pragma unroll
        for (int kb = 0; kb < K / 32; ++kb)
#pragma unroll
            for (int i = 0; i < 8; ++i) h[kb][i] = load2(hp + (32 * kb + i) * V);
    }
#pragma unroll
    for (int t = 0; t < TURNS; ++t) {
        const int at = t * NTHREADS + threadIdx.x, i = at / CHUNKS, d = at % CHUNKS;
        if (TURNS * NTHREADS == 16 * NT * CHUNKS || i < 16 * NT) {
            *reinterpret_cast<V16 *>(smem + L::k + i * L::ROWB + 16 * d) = kx[t];
            *reinterpret_cast<V16 *>(smem + L::q + i * L::ROWB + 16 * d) = qx[t];
        }
    }
    if (w == 0) {
        // path sums and ancestors by pointer doubling: after a round a lane has its sum
        // over twice as many nodes.  The sums are in 64 bits (their differences would lose
        // a small gate next to a large one), and e^g below 2^-149 is zero, so that a floor
        // under g keeps the differences finite where g is -inf.
        int at = up >= 0 && up < l ? up : -1;
        uint64_t m = at >= 0 ? 1ull << at : 0;
        double s = gate < -200.f ? -200.0 : (double)gate;
        while (__ballot(at >= 0)) {
            const int from = at < 0 ? l : at;
            const uint64_t pm = __shfl(m, from);
            const double ps = __shfl(s, from);
            const int pa = __shfl(at, from);
            if (at >= 0) {
                m |= pm;
                s += ps;
                at = pa;
            }
        }
        if (l < 16 * NT) {
            G[l] = s;
            mask[l] = m;
            eg[l] = expf((float)s);
            beta[l] = b;
        }
        if (l < 2) bad[l] = 0;
    }
    lds_barrier();

    auto row = [&](int base, int i, int kb) { return smem + base + i * L::ROWB + (32 * kb + 8 * g) * (int)sizeof(In); };
    // tiles of A and P, dealt to the waves
    int turn = 0;
#pragma unroll
    for (int rt = 0; rt < NT; ++rt)
#pragma unroll
        for (int ct = 0; ct <= rt; ++ct, ++turn) {
            if (turn % NW != w || rt >= nt) continue;
            f32x4 kk = zero4(), qk = zero4();
#pragma unroll
            for (int kb = 0; kb < K / 32; ++kb) {
                Row8<In> kr, qr, kc;
                kr.load(row(L::k, 16 * rt + c, kb));
                qr.load(row(L::q, 16 * rt + c, kb));
                kc.load(row(L::k, 16 * ct + c, kb));
                kk = kr.dot(kc, kk);
                qk = qr.dot(kc, qk);
            }
            const int jc = 16 * ct + c;  // the column's node
            const double Gc = G[jc];
            unsigned lost = 0;  // rows of this lane group's four that are not finite
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int i = 16 * rt + 4 * g + r;
                const bool above = mask[i] >> jc & 1;
                const float d = above ? expf((float)(G[i] - Gc)) : 0.f;
                float a = above ? beta[i] * d * kk[r] : 0.f;
                // a product of a row with itself shows whether it is finite
                if (!finite(a) || (i == jc && !finite(kk[r]))) {
                    lost |= 1u << r;
                    a = 0.f;
                }
                At[tile_at(rt, ct) + (4 * g + r) * LDT + c] = -a;
                Pt[tile_at(rt, ct) + (4 * g + r) * LDT + c] = above ? d * qk[r] : i == jc ? qk[r] : 0.f;
            }
            if (lost) atomicOr(&bad[rt >> 1], lost << (16 * (rt & 1) + 4 * g));
        }
    lds_barrier();
    // inverses of the diagonal tiles of I + A, a column per lane, in place
#pragma unroll
    for (int rt = 0; rt < NT; ++rt) {
        if (rt % NW != w || rt >= nt) continue;
        float *tile = At + tile_at(rt, rt);
        float x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = i == c ? 1.f : 0.f;
#pragma unroll
        for (int i = 1; i < 16; ++i) {
            f32x4 a[4];
#pragma unroll
            for (int m = 0; m <= (i - 1) / 4; ++m) a[m] = *reinterpret_cast<const f32x4 *>(tile + i * LDT + 4 * m);
#pragma unroll
            for (int m = 0; m < i; ++m) x[i] += a[m / 4][m % 4] * x[m];
        }
        if (g == 0)
#pragma unroll
            for (int i = 0; i < 16; ++i) tile[i * LDT + c] = x[i];
    }
    // K h and Q h
    f32x4 kh[NT][2], qh[NT][2];
#pragma unroll
    for (int rt = 0; rt < NT; ++rt)
#pragma unroll
        for (int t = 0; t < 2; ++t) kh[rt][t] = qh[rt][t] = zero4();
#pragma unroll
    for (int kb = 0; kb < K / 32; ++kb) {
        State8<In, PIECES> s[2];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            float x[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = h[kb][i][t];
            s[t].set(x);
        }
#pragma unroll
        for (int rt = 0; rt < NT; ++rt) {
            if (rt >= nt) continue;
            Row8<In> kr, qr;
            kr.load(row(L::k, 16 * rt + c, kb));
            qr.load(row(L::q, 16 * rt + c, kb));
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                kh[rt][t] = s[t].dot(kr, kh[rt][t]);
                qh[rt][t] = s[t].dot(qr, qh[rt][t]);
            }
        }
    }
    lds_barrier();
    const In *vp = reinterpret_cast<const In *>(p.v) + hv * V + col;
    uint64_t lost[2] = {0, 0};  // nodes whose right-hand side in this lane's columns is not finite
    f32x4 u[NT][2];
#pragma unroll
    for (int rt = 0; rt < NT; ++rt) {
        if (rt >= nt) continue;
        f32x4 r[2];
        const f32x4 e4 = *reinterpret_cast<const f32x4 *>(eg + 16 * rt + 4 * g);
        const f32x4 b4 = *reinterpret_cast<const f32x4 *>(beta + 16 * rt + 4 * g);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int node = 16 * rt + 4 * g + i;
            pair v = {0.f, 0.f};
            if (node < n) v = load2(vp + row_offset(p, j, bos + node, p.v_batch, p.v_row));
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                float x = b4[i] * (v[t] - e4[i] * kh[rt][t][i]);
                if (!finite(x)) {
                    lost[t] |= 1ull << node;
                    x = 0.f;
                }
                r[t][i] = x;
            }
        }
#pragma unroll
        for (int t = 0; t < 2; ++t) {
#pragma unroll
            for (int ct = 0; ct < rt; ++ct) r[t] = tile_mul(At + tile_at(rt, ct), u[ct][t], r[t]);
            u[rt][t] = tile_mul(At + tile_at(rt, rt), r[t], zero4());
        }
    }
    const uint64_t rows_lost = bad[0] | (uint64_t)bad[1] << 32;
    const bool poisoned = __ballot((lost[0] | lost[1] | rows_lost) != 0) != 0;
    if (poisoned)
#pragma unroll
        for (int t = 0; t < 2; ++t) {  // the column's nodes of all lane groups
            lost[t] |= rows_lost;
            lost[t] |= __shfl_xor(lost[t], 16);
            lost[t] |= __shfl_xor(lost[t], 32);
        }
#pragma unroll
    for (int rt = 0; rt < NT; ++rt) {
        if (rt >= nt) continue;
        const f32x4 e4 = *reinterpret_cast<const f32x4 *>(eg + 16 * rt + 4 * g);
        f32x4 y[2];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            y[t] = e4 * qh[rt][t];
#pragma unroll
            for (int ct = 0; ct <= rt; ++ct) y[t] = tile_mul(Pt + tile_at(rt, ct), u[ct][t], y[t]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int node = 16 * rt + 4 * g + i;
            pair x = {p.scale * y[0][i], p.scale * y[1][i]};
            if (poisoned) {
                const uint64_t path = mask[node] | 1ull << node;
                if (path & lost[0]) x[0] = __builtin_nanf("");
                if (path & lost[1]) x[1] = __builtin_nanf("");
            }
            if (node < n) store2(o + (bos + node) * p.Hv * V + col, x);
        }
    }
}

template <typename In, typename Out, int K, int V, int NT> hipError_t launch(const PoolParams &p, hipStream_t s) {
    constexpr int bytes = TreeLds<In, K, NT>::bytes;
    static const hipError_t attr =
        hipFuncSetAttribute(reinterpret_cast<const void *>(&gdr_tree_kernel<In, Out, K, V, NT>),
                            hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
    (void)attr;  // a refusal shows up as a launch error below
    launch_k(gdr_tree_kernel<In, Out, K, V, NT>, dim3((uint32_t)p.n_seq * p.Hv), dim3(2 * V), bytes, s, p);
    return hipGetLastError();
}

template <typename In, typename Out, int NT> hipError_t launch_kv(int K, int V, const PoolParams &p, hipStream_t s) {
    if (K == 128) return V == 128 ? launch<In, Out, 128, 128, NT>(p, s) : launch<In, Out, 128, 64, NT>(p, s);
    return V == 128 ? launch<In, Out, 64, 128, NT>(p, s) : launch<In, Out, 64, 64, NT>(p, s);
}

template <typename In, typename Out>
hipError_t launch_nt(int K, int V, int most, const PoolParams &p, hipStream_t s) {
    return most <= 16   ? launch_kv<In, Out, 1>(K, V, p, s)
           : most <= 32 ? launch_kv<In, Out, 2>(K, V, p, s)
                        : launch_kv<In, Out, 4>(K, V, p, s);
}

}  // namespace

hipError_t launch_tree(Dt dt, Dt out, int K, int V, int most, const PoolParams &p, hipStream_t s) {
    if (dt == Dt::BF16)
        return out == Dt::BF16 ? launch_nt<bf16, bf16>(K, V, most, p, s) : launch_nt<bf16, float>(K, V, most, p, s);
    return out == Dt::BF16 ? launch_nt<float, bf16>(K, V, most, p, s) : launch_nt<float, float>(K, V, most, p, s);
}

}  // namespace gdr
