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
// Only O is wanted, so U is never formed: with M (I + A) = P,
//     O = scale (e^G Q h + M R),   R = beta (V - e^G K h),
// and M, a matrix of nodes by nodes, is the same for all value columns.
//
// One workgroup per (sequence, v head), one wave per 32 value columns, nodes in
// NT tiles of 16.  The state is read once, straight into the registers that feed
// the products: lane (c, g) = (l & 15, l >> 4) of a wave loads h[32 kb + 8 g + i][2 c
// + t], the B operands of two 16-column tiles whose columns are 2 c and 2 c + 1.
// These loads are issued first and are in flight while the waves share out A and
// P (from K and Q in LDS).  A wave that has P's tiles of rows r in registers, transposed,
// solves M's rows r from the right: M^T_c = D_c^T (P^T_c + sum over k > c of (-A_kc)^T M^T_k), D
// the inverses of I + A's diagonal tiles.  An accumulator tile of M^T is an A operand
// tile of M, so M goes to LDS as it stands (in the place of K and Q), in bf16 pieces.
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

template <typename In, int K, int NT, int PIECES> struct TreeLds {
    static constexpr int ROWB = K * sizeof(In) + 16;  // a row of K or Q with padding
    static constexpr int TILES = NT * (NT + 1) / 2, NP = (NT + 1) / 2;
    static constexpr int k = 0, q = k + 16 * NT * ROWB, a = q + 16 * NT * ROWB, G = a + TILES * 16 * LDT * 4,
                         mask = G + 16 * NT * 8, eg = mask + 16 * NT * 8, beta = eg + 16 * NT * 4,
                         bad = beta + 16 * NT * 4, bytes = bad + 16;
    // M, in the place of K and Q: per row tile r, pairs of column tiles, piece and lane, 16 bytes
    static constexpr int m = 0, PAIR = PIECES * 1024;
    static __device__ __forceinline__ int pair_at(int r, int cp) { return m + ((r + 1) / 2 * (r / 2 + 1) + cp) * PAIR; }
    static_assert(((NT + 1) / 2 * (NT / 2 + 1)) * PAIR <= a, "M fits in the place of K and Q");
};

__device__ __forceinline__ bool finite4(f32x4 x) {
    return fmaxf(fmaxf(fabsf(x[0]), fabsf(x[1])), fmaxf(fabsf(x[2]), fabsf(x[3]))) < __builtin_inff() &&
           x[0] == x[0] && x[1] == x[1] && x[2] == x[2] && x[3] == x[3];
}
// tile (r, c) of a lower triangle of 16 x 16 tiles
__device__ __forceinline__ int tile_at(int r, int c) { return (r * (r + 1) / 2 + c) * 16 * LDT; }

// fp32 product of the transpose of a 16 x 16 tile of LDS and an accumulator tile
__device__ __forceinline__ f32x4 tile_t_mul(const float *tile, f32x4 b, f32x4 c) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
        c = __builtin_amdgcn_mfma_f32_16x16x4f32(tile[(4 * lg4() + j) * LDT + ln16()], b[j], c, 0, 0, 0);
    return c;
}

// x as a sum of bf16 values: 3 keep 24 bits (an fp32 output), 2 keep 16 (a bf16 output has 8)
template <int PIECES> __device__ __forceinline__ void pieces4(f32x4 x, bf16x4 *y) {
#pragma unroll
    for (int s = 0; s < PIECES; ++s) {
        y[s] = __builtin_convertvector(x, bf16x4);
        x -= __builtin_convertvector(y[s], f32x4);
    }
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

// eight state values of a column as an operand, in bf16 pieces where the rows are bf16
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
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// A buffer of n rows, `stride` bytes apart, of `bytes` bytes each: loads past its end give
// zero and stores there are dropped, so that rows need no conditions
typedef __amdgpu_buffer_rsrc_t Rsrc;
__device__ __forceinline__ Rsrc rows_of(const void *base, int n, int stride, int bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(base), 0, (n - 1) * stride + bytes, 0x00027000);
}
__device__ __forceinline__ void store2(float, Rsrc r, int lane, int at, pair x) {
    __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(u32x2, x), r, lane, at, 0);
}
__device__ __forceinline__ void store2(bf16, Rsrc r, int lane, int at, pair x) {
    __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, __builtin_convertvector(x, bf16x2)), r, lane, at, 0);
}

// waves per SIMD that the registers leave room for: what the LDS of NT = 4 leaves room for too
template <typename In, int V, int NT> constexpr int waves_per_simd() {
    return NT < 4 ? 3 : sizeof(In) == 4 ? 1 : V == 64 ? 2 : 3;
}

template <typename In, typename Out, int K, int V, int NT>
__global__ __launch_bounds__(2 * V, (waves_per_simd<In, V, NT>())) void gdr_tree_kernel(PoolParams p) {
    constexpr int NTHREADS = 2 * V, NW = V / 32, PIECES = sizeof(Out) == 4 ? 3 : 2;
    using L = TreeLds<In, K, NT, PIECES>;
    constexpr int NP = L::NP;
    extern __shared__ __align__(16) char smem[];
    float *At = reinterpret_cast<float *>(smem + L::a);  // -A, later with D in the diagonal tiles
    double *G = reinterpret_cast<double *>(smem + L::G);
    uint64_t *mask = reinterpret_cast<uint64_t *>(smem + L::mask);
    float *eg = reinterpret_cast<float *>(smem + L::eg), *beta = reinterpret_cast<float *>(smem + L::beta);
    unsigned *bad = reinterpret_cast<unsigned *>(smem + L::bad);  // two words of node bits

    const int unit = xcd_runs(blockIdx.x, gridDim.x), j = unit / p.Hv, hv = unit - j * p.Hv, hq = hv / (p.Hv / p.Hq);
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

    // wave 0: parents, gates and beta, a node per lane
    int up = -1;
    float gate = 0.f, b = 0.f;
    if (w == 0 && l < n) {
        up = p.parents[bos + l];
        gate = p.g[(bos + l) * p.Hv + hv];
        b = p.beta[(bos + l) * p.Hv + hv];
    }
    // K and Q; rows past the last node read as zero (or, where rows overlap, as any values:
    // nothing below depends on them)
    constexpr int PER = Vec16<In>::n, CHUNKS = K / PER, ROWS = NTHREADS / CHUNKS, TURNS = 16 * NT / ROWS > 0 ? 16 * NT / ROWS : 1;
    static_assert(NTHREADS % CHUNKS == 0 && ((16 * NT) % ROWS == 0 || ROWS > 16 * NT), "whole turns");
    const int kq_row = threadIdx.x / CHUNKS, kq_chunk = threadIdx.x % CHUNKS;
    u32x4 kx[TURNS], qx[TURNS];
    {
        const int kb = (int)p.k_row * (int)sizeof(In), qb = (int)p.q_row * (int)sizeof(In);
        const Rsrc kr = rows_of(reinterpret_cast<const In *>(p.k) + row_offset(p, j, bos, p.k_batch, p.k_row) + hq * K, n, kb, K * sizeof(In));
        const Rsrc qr = rows_of(reinterpret_cast<const In *>(p.q) + row_offset(p, j, bos, p.q_batch, p.q_row) + hq * K, n, qb, K * sizeof(In));
#pragma unroll
        for (int t = 0; t < TURNS; ++t) {
            kx[t] = __builtin_amdgcn_raw_buffer_load_b128(kr, kq_row * kb + 16 * kq_chunk, t * ROWS * kb, 0);
            qx[t] = __builtin_amdgcn_raw_buffer_load_b128(qr, kq_row * qb + 16 * kq_chunk, t * ROWS * qb, 0);
        }
    }
    // the state and V
    pair h[K / 32][8];
    {
        const Rsrc hr = rows_of(p.states + (int64_t)slot * p.slot_stride + (int64_t)hv * K * V, K, 4 * V, 4 * V);
#pragma unroll
        for (int kb = 0; kb < K / 32; ++kb)
#pragma unroll
            for (int i = 0; i < 8; ++i)
                h[kb][i] = __builtin_bit_cast(pair, __builtin_amdgcn_raw_buffer_load_b64(hr, (8 * g * V + col) * 4, (32 * kb + i) * V * 4, 0));
    }
    typedef In InPair __attribute__((ext_vector_type(2)));
    InPair v[NT][4];
    {
        const int vb = (int)p.v_row * (int)sizeof(In);
        const Rsrc vr = rows_of(reinterpret_cast<const In *>(p.v) + row_offset(p, j, bos, p.v_batch, p.v_row) + hv * V, n, vb, V * sizeof(In));
#pragma unroll
        for (int rt = 0; rt < NT; ++rt)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int lane = 4 * g * vb + col * (int)sizeof(In), at = (16 * rt + i) * vb;
                if constexpr (sizeof(In) == 2)
                    v[rt][i] = __builtin_bit_cast(InPair, __builtin_amdgcn_raw_buffer_load_b32(vr, lane, at, 0));
                else
                    v[rt][i] = __builtin_bit_cast(InPair, __builtin_amdgcn_raw_buffer_load_b64(vr, lane, at, 0));
            }
    }
#pragma unroll
    for (int t = 0; t < TURNS; ++t)
        if (ROWS <= 16 * NT || kq_row < 16 * NT) {
            *reinterpret_cast<u32x4 *>(smem + L::k + (t * ROWS + kq_row) * L::ROWB + 16 * kq_chunk) = kx[t];
            *reinterpret_cast<u32x4 *>(smem + L::q + (t * ROWS + kq_row) * L::ROWB + 16 * kq_chunk) = qx[t];
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
    // products of the nodes of tile a (rows) with those of tile b (columns); lane (c, g) then
    // has nodes 16 a + 4 g + i against node 16 b + c
    auto product = [&](int a, int base_b, int b) {
        f32x4 x = zero4();
#pragma unroll
        for (int kb = 0; kb < K / 32; ++kb) {
            Row8<In> ra, rb;
            ra.load(row(L::k, 16 * a + c, kb));
            rb.load(row(base_b, 16 * b + c, kb));
            x = ra.dot(rb, x);
        }
        return x;
    };
    // D of node 16 b + c and its ancestors among nodes 16 a + 4 g + i, zero for the others
    auto decay = [&](int a, double Gb, uint64_t mb) {
        f32x4 d;
        const uint32_t bits = (uint32_t)(mb >> (16 * a + 4 * g));
#pragma unroll
        for (int i = 0; i < 4; ++i) d[i] = bits >> i & 1 ? fast_exp((float)(Gb - G[16 * a + 4 * g + i])) : 0.f;
        return d;
    };
    // a wave takes P's rows r and, so that all waves have as many tiles, A's rows NT - 1 - r
    constexpr int MINE = NT > NW ? NT / NW : 1;
    f32x4 mt[MINE][NT];
#pragma unroll
    for (int y = 0; y < MINE; ++y) {
        const int r = y ? NT - 1 - w : w, ra = NT - 1 - r;
        if (r >= NT) break;
        if (ra < nt) {
            const int node = 16 * ra + c;
            const double Gb = G[node];
            const uint64_t mb = mask[node];
            const float minus_beta = -beta[node];
            bool lost = false;
#pragma unroll
            for (int ct = 0; ct < NT; ++ct) {
                if (ct > ra) continue;
                const f32x4 kk = product(ct, L::k, ra), d = decay(ct, Gb, mb);
                f32x4 a;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    a[i] = d[i] != 0.f ? minus_beta * d[i] * kk[i] : 0.f;
                    // a product of a row with itself shows whether it is finite
                    if (16 * ct + 4 * g + i == node) lost |= !(fabsf(kk[i]) < __builtin_inff());
                }
                if (!finite4(a)) {
                    lost = true;
                    a = zero4();
                }
                *reinterpret_cast<f32x4 *>(At + tile_at(ra, ct) + c * LDT + 4 * g) = a;
            }
            if (lost) atomicOr(&bad[ra >> 1], 1u << (16 * (ra & 1) + c));
        }
        if (r < nt) {
            const int node = 16 * r + c;
            const double Gb = G[node];
            const uint64_t mb = mask[node] | 1ull << node;
#pragma unroll
            for (int ct = 0; ct < NT; ++ct) {
                mt[y][ct] = zero4();
                if (ct > r) continue;
                const f32x4 kq = product(ct, L::q, r), d = decay(ct, Gb, mb);
#pragma unroll
                for (int i = 0; i < 4; ++i) mt[y][ct][i] = d[i] != 0.f ? d[i] * kq[i] : 0.f;
            }
        }
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
    // M's rows r, from the right; the products with K and Q are done, M takes their place
#pragma unroll
    for (int y = 0; y < MINE; ++y) {
        const int r = y ? NT - 1 - w : w;
        if (r >= nt) break;
#pragma unroll
        for (int ct = NT - 1; ct >= 0; --ct) {
            if (ct > r) continue;
#pragma unroll
            for (int k = ct + 1; k < NT; ++k)
                if (k <= r) mt[y][ct] = tile_t_mul(At + tile_at(k, ct), mt[y][k], mt[y][ct]);
            mt[y][ct] = tile_t_mul(At + tile_at(ct, ct), mt[y][ct], zero4());
        }
#pragma unroll
        for (int cp = 0; cp < NP; ++cp) {
            if (2 * cp > r) continue;
            bf16x4 lo[PIECES], hi[PIECES];
            pieces4<PIECES>(mt[y][2 * cp], lo);
            pieces4<PIECES>(2 * cp + 1 < NT ? mt[y][2 * cp + 1 < NT ? 2 * cp + 1 : 0] : zero4(), hi);  // zero past r
#pragma unroll
            for (int s = 0; s < PIECES; ++s)
                *reinterpret_cast<bf16x8 *>(smem + L::pair_at(r, cp) + 1024 * s + 16 * l) = cat(lo[s], hi[s]);
        }
    }
    // R, where not finite remembered and replaced
    uint64_t lost[2] = {0, 0};  // nodes, in this lane's columns
    bf16x8 rs[NP][2][PIECES];
#pragma unroll
    for (int cp = 0; cp < NP; ++cp) {
        bf16x4 half[2][2][PIECES];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int rt = 2 * cp + e;
            f32x4 x[2] = {zero4(), zero4()};
            if (rt < NT && rt < nt) {
                const f32x4 e4 = *reinterpret_cast<const f32x4 *>(eg + 16 * rt + 4 * g);
                const f32x4 b4 = *reinterpret_cast<const f32x4 *>(beta + 16 * rt + 4 * g);
#pragma unroll
                for (int t = 0; t < 2; ++t) {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        x[t][i] = b4[i] * (to_f32(v[rt < NT ? rt : 0][i][t]) - e4[i] * kh[rt < NT ? rt : 0][t][i]);
                    if (!finite4(x[t]))
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (!(fabsf(x[t][i]) < __builtin_inff())) {
                                lost[t] |= 1ull << (16 * rt + 4 * g + i);
                                x[t][i] = 0.f;
                            }
                }
            }
#pragma unroll
            for (int t = 0; t < 2; ++t) pieces4<PIECES>(x[t], half[e][t]);
        }
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int s = 0; s < PIECES; ++s) rs[cp][t][s] = cat(half[0][t][s], half[1][t][s]);
    }
    lds_barrier();
    const int ob = p.Hv * V * (int)sizeof(Out);
    const Rsrc out = rows_of(o + bos * p.Hv * V, n, ob, V * sizeof(Out));
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
        for (int t = 0; t < 2; ++t) y[t] = e4 * qh[rt][t];
#pragma unroll
        for (int cp = 0; cp <= rt / 2; ++cp) {
            bf16x8 m[PIECES];
#pragma unroll
            for (int s = 0; s < PIECES; ++s)
                m[s] = *reinterpret_cast<const bf16x8 *>(smem + L::pair_at(rt, cp) + 1024 * s + 16 * l);
            // the products that PIECES pieces of accuracy need, small ones first
#pragma unroll
            for (int sum = PIECES - 1; sum >= 0; --sum)
#pragma unroll
                for (int s = 0; s <= sum; ++s)
#pragma unroll
                    for (int t = 0; t < 2; ++t)
                        y[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(m[s], rs[cp][t][sum - s], y[t], 0, 0, 0);
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
            store2(Out(), out, 4 * g * ob + col * (int)sizeof(Out), (16 * rt + i) * ob, x);
        }
    }
}

template <typename In, typename Out, int K, int V, int NT> hipError_t launch(const PoolParams &p, hipStream_t s) {
    constexpr int bytes = TreeLds<In, K, NT, sizeof(Out) == 4 ? 3 : 2>::bytes;
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
