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
// tile of M, so M goes to LDS as it stands (in the place of K and Q), in bf16 pieces.  The last
// product is of 2 M and R / 2: from 2^128 - 2^119 on the first piece of a finite value of R
// would be infinite, and NaN against the zeros of other nodes' rows of M.
// fp32 rows of K and Q are split into pieces on their way to LDS: 8 trees of 64 nodes (fp32,
// K = V = 128) take 17.0 us, 22.4 with fp32 matrix instructions, 13.0 with bf16 rows.
//
// 64 packed trees of 37 to 64 nodes (H_v = 32, K = V = 128, bf16; 214 MB) take 54.5 us, 3.9 TB/s,
// where a large copy runs at 5.0: three workgroups per compute unit hide most of their phases
// from each other, but not all (two per unit take 2 us more), and the matrix units are busy for
// 30% of it.  Small batches are bound by the chain of phases: one tree of 13 nodes takes 6.3 us,
// of 64 nodes 11.7.  Of the 23,000 cycles of a lone workgroup of 64 nodes, 5,500 pass until K and Q
// are in LDS, the tiles of A and P take 3,000, D 2,000, K h and Q h 5,900, M 2,600, R 1,600 and
// the output 2,700.  With two pieces (see PIECES) persistent workgroups with the next tree's loads
// in flight took 75 us where this form took 49, tiles chosen by runtime conditions, each a branch
// of its own, 54.6 against 52, U by forward substitution in every wave instead of M 101 against
// 60.5.
//
// Non-finite values.  Node j must not reach nodes that are no descendants of it,
// though a product with a masked zero would turn its NaN or infinity into NaN there.
// Products by rows keep to their rows; entries of A and of D (products of A's entries, which
// may overflow where these are finite) and right-hand sides that are not finite are replaced
// by zero and remembered (by node, or by node and column), and the rows of those nodes and of
// their descendants are written as NaN.
#include "gdr_lds.hpp"
#include "gdr_pool.hpp"

namespace gdr {
namespace {

constexpr int LDT = 20;  // floats per row of a 16 x 16 tile in LDS (16 and padding: conflict-free rows)
// bf16 pieces of an fp32 value: 3 keep its 24 bits, with a bf16 output too.  There 2 (16 bits)
// would take 8 us less for the 64 packed trees above and 0.4 less for one tree of 13 nodes,
// but lose what is small by cancellation, which fp32 products keep
constexpr int PIECES = 3;

template <typename In, int K, int NT> struct TreeLds {
    // K and Q: a plane of bf16 rows (with padding) per piece, one where they are bf16
    static constexpr int ROWB = 2 * K + 16, PLANE = 16 * NT * ROWB, PLANES = sizeof(In) == 2 ? 1 : PIECES;
    static constexpr int TILES = NT * (NT + 1) / 2, NP = (NT + 1) / 2;
    static constexpr int k = 0, q = k + PLANES * PLANE, a = q + PLANES * PLANE, G = a + TILES * 16 * LDT * 4,
                         mask = G + 16 * NT * 8, eg = mask + 16 * NT * 8, beta = eg + 16 * NT * 4,
                         bad = beta + 16 * NT * 4, bytes = bad + 16;
    // M, in the place of K and Q: per row tile r, pairs of column tiles, piece and lane, 16 bytes
    static constexpr int m = 0, PAIR = PIECES * 1024;
    static __device__ __forceinline__ int pair_at(int r, int cp) { return m + ((r + 1) / 2 * (r / 2 + 1) + cp) * PAIR; }
    static_assert(((NT + 1) / 2 * (NT / 2 + 1)) * PAIR <= a, "M fits in the place of K and Q");
};

// tile (r, c) of a lower triangle of 16 x 16 tiles
__device__ __forceinline__ int tile_at(int r, int c) { return (r * (r + 1) / 2 + c) * 16 * LDT; }

// fp32 product of the transpose of a 16 x 16 tile of LDS and an accumulator tile
__device__ __forceinline__ f32x4 tile_t_mul(const float *tile, f32x4 b, f32x4 c) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
        c = __builtin_amdgcn_mfma_f32_16x16x4f32(tile[(4 * lg4() + j) * LDT + ln16()], b[j], c, 0, 0, 0);
    return c;
}

// two values as sums of bf16 ones
__device__ __forceinline__ void pieces2(float a, float b, uint32_t *y) {
#pragma unroll
    for (int s = 0; s < PIECES; ++s) {
        y[s] = __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{a, b}, bf16x2));
        a -= __builtin_bit_cast(float, y[s] << 16);
        b -= __builtin_bit_cast(float, y[s] & 0xffff0000u);
    }
}
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
// eight values, an operand's, in pieces
__device__ __forceinline__ void pieces8(f32x4 x, f32x4 y, bf16x8 *z) {
    uint32_t a[4][PIECES];
    pieces2(x[0], x[1], a[0]);
    pieces2(x[2], x[3], a[1]);
    pieces2(y[0], y[1], a[2]);
    pieces2(y[2], y[3], a[3]);
#pragma unroll
    for (int s = 0; s < PIECES; ++s) z[s] = __builtin_bit_cast(bf16x8, (u32x4{a[0][s], a[1][s], a[2][s], a[3][s]}));
}

// Eight consecutive values of a row of K or Q (P = 1 piece, or PIECES of fp32 values), or of
// a state column (PIECES), and their product as a sequence of matrix instructions that is
// taken step by step over several tiles, so that none waits for another.
template <int P> struct Eight {
    bf16x8 x[P];
    // a row in planes `plane` bytes apart
    __device__ __forceinline__ void load(const char *p, int plane) {
#pragma unroll
        for (int s = 0; s < P; ++s) x[s] = *reinterpret_cast<const bf16x8 *>(p + s * plane);
    }
};
// steps of a product of A and B pieces: those that `keep` pieces of accuracy need
constexpr int steps(int A, int B, int keep) {
    int n = 0;
    for (int s = 0; s < A; ++s)
        for (int z = 0; z < B; ++z) n += s + z < keep;
    return n;
}
// the s-th one, small ones first
template <int KEEP, int A, int B>
__device__ __forceinline__ f32x4 product_step(int step, const Eight<A> &a, const Eight<B> &b, f32x4 c) {
    int n = 0;
#pragma unroll
    for (int sum = KEEP - 1; sum >= 0; --sum)
#pragma unroll
        for (int s = 0; s < A; ++s) {
            if (sum - s < 0 || sum - s >= B) continue;
            if (n++ == step) return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.x[s], b.x[sum - s], c, 0, 0, 0);
        }
    return c;
}

typedef float pair __attribute__((ext_vector_type(2)));

// A buffer of n rows, `stride` bytes apart, of `bytes` bytes each: loads past its end give
// zero and stores there are dropped, so that rows need no conditions.  (Where that can
// happen the whole offset is the lane's, the part that is always compared with the end.)
typedef __amdgpu_buffer_rsrc_t Rsrc;
constexpr int ONCE = 2;  // nontemporal: the state and the output, which pass by once
__device__ __forceinline__ Rsrc rows_of(const void *base, int n, int stride, int bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(base), 0, (n - 1) * stride + bytes, 0x00027000);
}
__device__ __forceinline__ void store2(float, Rsrc r, int at, pair x) {
    __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(u32x2, x), r, at, 0, ONCE);
}
__device__ __forceinline__ void store2(bf16, Rsrc r, int at, pair x) {
    __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, __builtin_convertvector(x, bf16x2)), r, at, 0, ONCE);
}

// One tree of n nodes, up to 16 NT, and one v head; every wave of the workgroup calls it.
template <typename In, typename Out, int K, int V, int NT>
__device__ __forceinline__ void tree(const PoolParams &p, char *smem, int j, int hv, int64_t bos, int n) {
    constexpr int NTHREADS = 2 * V, NW = V / 32;
    using L = TreeLds<In, K, NT>;
    typedef Eight<L::PLANES> Row;
    constexpr int NP = L::NP;
    float *At = reinterpret_cast<float *>(smem + L::a);  // -A, later with D in the diagonal tiles
    double *G = reinterpret_cast<double *>(smem + L::G);
    uint64_t *mask = reinterpret_cast<uint64_t *>(smem + L::mask);
    float *eg = reinterpret_cast<float *>(smem + L::eg), *half_beta = reinterpret_cast<float *>(smem + L::beta);
    unsigned *bad = reinterpret_cast<unsigned *>(smem + L::bad);  // two words of node bits
    const int l = lane_id(), w = __builtin_amdgcn_readfirstlane(wave_id()), c = ln16(), g = lg4();
    const int col = 32 * w + 2 * c, hq = hv / (p.Hv / p.Hq);

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
    constexpr int PER = Vec16<In>::n, CHUNKS = K / PER, ROWS = NTHREADS / CHUNKS, TURNS = (16 * NT + ROWS - 1) / ROWS;
    const int kq_row = threadIdx.x / CHUNKS, kq_chunk = threadIdx.x % CHUNKS;
    u32x4 kx[TURNS], qx[TURNS];
    {
        const int kb = (int)p.k_row * (int)sizeof(In), qb = (int)p.q_row * (int)sizeof(In);
        const Rsrc kr = rows_of(reinterpret_cast<const In *>(p.k) + row_offset(p, j, bos, p.k_batch, p.k_row) + hq * K, n,
                                kb, K * sizeof(In));
        const Rsrc qr = rows_of(reinterpret_cast<const In *>(p.q) + row_offset(p, j, bos, p.q_batch, p.q_row) + hq * K, n,
                                qb, K * sizeof(In));
#pragma unroll
        for (int t = 0; t < TURNS; ++t) {
            kx[t] = __builtin_amdgcn_raw_buffer_load_b128(kr, (t * ROWS + kq_row) * kb + 16 * kq_chunk, 0, 0);
            qx[t] = __builtin_amdgcn_raw_buffer_load_b128(qr, (t * ROWS + kq_row) * qb + 16 * kq_chunk, 0, 0);
        }
    }
    const int ob = p.Hv * V * (int)sizeof(Out);
    const Rsrc out = rows_of(reinterpret_cast<Out *>(p.o) + (bos * p.Hv + hv) * V, n, ob, V * sizeof(Out));
    const int slot = slot_of(p, j);
    if (slot < 0) {
#pragma unroll
        for (int i = 0; i < 4 * NT; ++i)
            store2(Out(), out, (16 * (i / 4) + 4 * g + i % 4) * ob + col * (int)sizeof(Out), pair{0.f, 0.f});
        return;
    }
    // the state, whose slot is looked up only now
    pair h[K / 32][8];
    {
        const Rsrc hr = rows_of(p.states + (int64_t)slot * p.slot_stride + (int64_t)hv * K * V, K, 4 * V, 4 * V);
#pragma unroll
        for (int kb = 0; kb < K / 32; ++kb)
#pragma unroll
            for (int i = 0; i < 8; ++i)
                h[kb][i] = __builtin_bit_cast(
                    pair, __builtin_amdgcn_raw_buffer_load_b64(hr, (8 * g * V + col) * 4, (32 * kb + i) * V * 4, ONCE));
    }
#pragma unroll
    for (int t = 0; t < TURNS; ++t)
        if (16 * NT % ROWS == 0 || t * ROWS + kq_row < 16 * NT) {
            char *to = smem + L::k + (t * ROWS + kq_row) * L::ROWB + 2 * PER * kq_chunk;
            if constexpr (sizeof(In) == 2) {
                *reinterpret_cast<u32x4 *>(to) = kx[t];
                *reinterpret_cast<u32x4 *>(to + L::q) = qx[t];
            } else {
#pragma unroll
                for (int kq = 0; kq < 2; ++kq) {
                    const f32x4 x = __builtin_bit_cast(f32x4, kq ? qx[t] : kx[t]);
                    uint32_t lo[PIECES], hi[PIECES];
                    pieces2(x[0], x[1], lo);
                    pieces2(x[2], x[3], hi);
#pragma unroll
                    for (int s = 0; s < PIECES; ++s)
                        *reinterpret_cast<u32x2 *>(to + kq * L::q + s * L::PLANE) = u32x2{lo[s], hi[s]};
                }
            }
        }
    if (w == 0) {
        // path sums and ancestors by pointer doubling: after a round a lane has its sum
        // over twice as many nodes.  The sums are in 64 bits (their differences would lose
        // a small gate next to a large one), and e^g below 2^-149 is zero, so that a floor
        // under g keeps the differences finite where g is -inf.  Later gates cannot lift what
        // the floor stands for: its node is their ancestor, and from more than 88 between the
        // two on, D is infinite and the row NaN anyway (-200 + 88 still has an e^ of zero).
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
            half_beta[l] = 0.5f * b;
        }
        if (l < 2) bad[l] = 0;
    }
    lds_barrier();

    auto load = [&](Row &x, int base, int i, int kb) { x.load(smem + base + i * L::ROWB + (32 * kb + 8 * g) * 2, L::PLANE); };
    // Rows r of A and of 2 P, transposed: lane (c, g) has node 16 r + c against nodes
    // 16 ct + 4 g + i, whose decay D both share.  Tiles past the diagonal come out zero.
    constexpr int MINE = (NT + NW - 1) / NW;
    f32x4 mt[MINE][NT];
#pragma unroll
    for (int y = 0; y < MINE; ++y) {
        const int r = w + y * NW;
        if (r >= NT) break;
        f32x4 kk[NT];
#pragma unroll
        for (int ct = 0; ct < NT; ++ct) kk[ct] = mt[y][ct] = zero4();
#pragma unroll
        for (int kb = 0; kb < K / 32; ++kb) {
            Row kr, qr, kc[NT];
            load(kr, L::k, 16 * r + c, kb);
            load(qr, L::q, 16 * r + c, kb);
#pragma unroll
            for (int ct = 0; ct < NT; ++ct) load(kc[ct], L::k, 16 * ct + c, kb);
#pragma unroll
            for (int s = 0; s < steps(L::PLANES, L::PLANES, L::PLANES); ++s)
#pragma unroll
                for (int ct = 0; ct < NT; ++ct) {
                    kk[ct] = product_step<L::PLANES>(s, kc[ct], kr, kk[ct]);
                    mt[y][ct] = product_step<L::PLANES>(s, kc[ct], qr, mt[y][ct]);
                }
            if constexpr (NT > 2) __builtin_amdgcn_sched_barrier(0);
        }
        const int node = 16 * r + c;
        const double Gb = G[node];
        const uint64_t above = mask[node];
        const float minus_beta = -2.f * half_beta[node];
        float probe = 0.f;  // becomes NaN where K's row or a row of A is not finite
#pragma unroll
        for (int ct = 0; ct < NT; ++ct) {
            const uint32_t bits = (uint32_t)(above >> (16 * ct + 4 * g));
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const bool self = 16 * ct + 4 * g + i == node, on = bits >> i & 1;
                const float d = fast_exp((float)(Gb - G[16 * ct + 4 * g + i]));
                if (self) probe += 0.f * kk[ct][i];
                kk[ct][i] = on ? minus_beta * d * kk[ct][i] : 0.f;
                probe += 0.f * kk[ct][i];
                mt[y][ct][i] = on || self ? 2.f * d * mt[y][ct][i] : 0.f;
            }
        }
        if (__ballot(probe != probe)) {
            if (probe != probe) atomicOr(&bad[r >> 1], 1u << (16 * (r & 1) + c));
#pragma unroll
            for (int ct = 0; ct < NT; ++ct)
#pragma unroll
                for (int i = 0; i < 4; ++i) kk[ct][i] = fabsf(kk[ct][i]) < __builtin_inff() ? kk[ct][i] : 0.f;
        }
#pragma unroll
        for (int ct = 0; ct < NT; ++ct)
            if (ct <= r) *reinterpret_cast<f32x4 *>(At + tile_at(r, ct) + c * LDT + 4 * g) = kk[ct];
    }
    // D, the inverses of the diagonal tiles of I + A, in place: a wave's own rows, a column per lane
#pragma unroll
    for (int y = 0; y < MINE; ++y) {
        const int r = w + y * NW;
        if (r >= NT) break;
        float *tile = At + tile_at(r, r);
        float x[16];
        // kept finite (med3 makes a NaN the least of the others), so that an entry past fp32's
        // range, found below by its size, meets a zero of A as zero.  (The substitution once
        // more in a branch of its own, without the zeros, made the registers spill: the 64 packed
        // trees took 84 us.)
        constexpr float MOST = __FLT_MAX__;
        float most = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = i == c ? 1.f : 0.f;
#pragma unroll
        for (int i = 1; i < 16; ++i) {
            f32x4 a[4];
#pragma unroll
            for (int m = 0; m <= (i - 1) / 4; ++m) a[m] = *reinterpret_cast<const f32x4 *>(tile + i * LDT + 4 * m);
#pragma unroll
            for (int m = 0; m < i; ++m) x[i] += a[m / 4][m % 4] * x[m];
            x[i] = __builtin_amdgcn_fmed3f(x[i], -MOST, MOST);
            most = fmaxf(most, fabsf(x[i]));
        }
        if (__ballot(most >= MOST)) {
            uint32_t over = 0;
#pragma unroll
            for (int i = 1; i < 16; ++i)
                if (fabsf(x[i]) >= MOST) {
                    over |= 1u << i;
                    x[i] = 0.f;
                }
            if (over) atomicOr(&bad[r >> 1], over << 16 * (r & 1));
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
        Eight<PIECES> s[2];
#pragma unroll
        for (int t = 0; t < 2; ++t)
            pieces8(f32x4{h[kb][0][t], h[kb][1][t], h[kb][2][t], h[kb][3][t]},
                            f32x4{h[kb][4][t], h[kb][5][t], h[kb][6][t], h[kb][7][t]}, s[t].x);
        // K's rows, then Q's: the rows of both at once would not leave the registers for a
        // third wave per SIMD
#pragma unroll
        for (int kq = 0; kq < 2; ++kq) {
            Row x[NT];
#pragma unroll
            for (int rt = 0; rt < NT; ++rt) load(x[rt], kq ? L::q : L::k, 16 * rt + c, kb);
#pragma unroll
            for (int step = 0; step < steps(L::PLANES, PIECES, PIECES); ++step)
#pragma unroll
                for (int rt = 0; rt < NT; ++rt)
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        f32x4 &y = kq ? qh[rt][t] : kh[rt][t];
                        y = product_step<PIECES>(step, x[rt], s[t], y);
                    }
            if constexpr (NT > 2) __builtin_amdgcn_sched_barrier(0);
        }
    }
    // V, in flight while M is solved (earlier, its registers would be missed)
    typedef In InPair __attribute__((ext_vector_type(2)));
    InPair v[NT][4];
    {
        const int vb = (int)p.v_row * (int)sizeof(In);
        const Rsrc vr = rows_of(reinterpret_cast<const In *>(p.v) + row_offset(p, j, bos, p.v_batch, p.v_row) + hv * V, n,
                                vb, V * sizeof(In));
#pragma unroll
        for (int rt = 0; rt < NT; ++rt)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int at = (16 * rt + 4 * g + i) * vb + col * (int)sizeof(In);
                if constexpr (sizeof(In) == 2)
                    v[rt][i] = __builtin_bit_cast(InPair, __builtin_amdgcn_raw_buffer_load_b32(vr, at, 0, 0));
                else
                    v[rt][i] = __builtin_bit_cast(InPair, __builtin_amdgcn_raw_buffer_load_b64(vr, at, 0, 0));
            }
    }
    lds_barrier();
    // 2 M's rows r, from the right; the products with K and Q are done, M takes their place
#pragma unroll
    for (int y = 0; y < MINE; ++y) {
        const int r = w + y * NW;
        if (r >= NT) break;
#pragma unroll
        for (int ct = NT - 1; ct >= 0; --ct) {
#pragma unroll
            for (int k = NT - 1; k > ct; --k) mt[y][ct] = tile_t_mul(At + tile_at(k, ct), mt[y][k], mt[y][ct]);
            mt[y][ct] = tile_t_mul(At + tile_at(ct, ct), mt[y][ct], zero4());
        }
#pragma unroll
        for (int cp = 0; cp < NP; ++cp) {
            bf16x8 m[PIECES];
            pieces8(mt[y][2 * cp], 2 * cp + 1 < NT ? mt[y][2 * cp + 1 < NT ? 2 * cp + 1 : 0] : zero4(), m);
            if (2 * cp <= r)
#pragma unroll
                for (int s = 0; s < PIECES; ++s)
                    *reinterpret_cast<bf16x8 *>(smem + L::pair_at(r, cp) + 1024 * s + 16 * l) = m[s];
        }
    }
    // R / 2, in the place of K h
    float probe = 0.f;
#pragma unroll
    for (int rt = 0; rt < NT; ++rt) {
        const f32x4 e4 = *reinterpret_cast<const f32x4 *>(eg + 16 * rt + 4 * g);
        const f32x4 b4 = *reinterpret_cast<const f32x4 *>(half_beta + 16 * rt + 4 * g);
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                kh[rt][t][i] = b4[i] * (to_f32(v[rt][i][t]) - e4[i] * kh[rt][t][i]);
                probe += 2.f * fabsf(kh[rt][t][i]);
            }
    }
    uint64_t lost[2] = {0, 0};  // nodes whose R in this lane's columns is not finite
    if (__ballot(!(probe < __builtin_inff())))
#pragma unroll
        for (int rt = 0; rt < NT; ++rt)
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (!(fabsf(kh[rt][t][i]) < 0x1p127f)) {
                        lost[t] |= 1ull << (16 * rt + 4 * g + i);
                        kh[rt][t][i] = 0.f;
                    }
    bf16x8 rs[NP][2][PIECES];
#pragma unroll
    for (int cp = 0; cp < NP; ++cp)
#pragma unroll
        for (int t = 0; t < 2; ++t)
            pieces8(kh[2 * cp][t], 2 * cp + 1 < NT ? kh[2 * cp + 1 < NT ? 2 * cp + 1 : 0][t] : zero4(), rs[cp][t]);
    lds_barrier();
    const uint64_t rows_lost = bad[0] | (uint64_t)bad[1] << 32;
    const bool poisoned = __ballot((lost[0] | lost[1] | rows_lost) != 0) != 0;
    f32x4 o[NT][2];
#pragma unroll
    for (int rt = 0; rt < NT; ++rt) {
        const f32x4 e4 = *reinterpret_cast<const f32x4 *>(eg + 16 * rt + 4 * g);
#pragma unroll
        for (int t = 0; t < 2; ++t) o[rt][t] = e4 * qh[rt][t];
    }
#pragma unroll
    for (int cp = 0; cp < NP; ++cp) {
        bf16x8 m[NT][PIECES];
#pragma unroll
        for (int rt = 2 * cp; rt < NT; ++rt)
#pragma unroll
            for (int s = 0; s < PIECES; ++s)
                m[rt][s] = *reinterpret_cast<const bf16x8 *>(smem + L::pair_at(rt, cp) + 1024 * s + 16 * l);
        // the products that PIECES pieces of accuracy need, small ones first
#pragma unroll
        for (int sum = PIECES - 1; sum >= 0; --sum)
#pragma unroll
            for (int s = 0; s <= sum; ++s)
#pragma unroll
                for (int rt = 2 * cp; rt < NT; ++rt)
#pragma unroll
                    for (int t = 0; t < 2; ++t)
                        o[rt][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(m[rt][s], rs[cp][t][sum - s], o[rt][t], 0, 0, 0);
    }
    if (poisoned) {
#pragma unroll
        for (int t = 0; t < 2; ++t) {  // the column's nodes of all lane groups
            lost[t] |= rows_lost;
            lost[t] |= __shfl_xor(lost[t], 16);
            lost[t] |= __shfl_xor(lost[t], 32);
#pragma unroll
            for (int rt = 0; rt < NT; ++rt)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int node = 16 * rt + 4 * g + i;
                    if ((mask[node] | 1ull << node) & lost[t]) o[rt][t][i] = __builtin_nanf("");
                }
        }
    }
#pragma unroll
    for (int rt = 0; rt < NT; ++rt)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            store2(Out(), out, (16 * rt + 4 * g + i) * ob + col * (int)sizeof(Out),
                   pair{p.scale * o[rt][0][i], p.scale * o[rt][1][i]});
}

// waves per SIMD that the registers (and, where NT = 4, LDS) leave room for
template <typename In, int V, int NT> constexpr int waves_per_simd() {
    return NT < 4 ? 3 : sizeof(In) == 4 ? 1 : V == 64 ? 2 : 3;
}

// trees of up to 16 NT nodes
template <typename In, typename Out, int K, int V, int NT>
__global__ __launch_bounds__(2 * V, (waves_per_simd<In, V, NT>())) void gdr_tree_kernel(PoolParams p) {
    extern __shared__ __align__(16) char smem[];
    const int unit = xcd_runs(blockIdx.x, gridDim.x), j = unit / p.Hv, hv = unit - j * p.Hv;
    int64_t bos, eos;
    token_range(p, j, bos, eos);
    const int64_t n = eos - bos;
    if (n <= 0) return;
    if (n > 16 * NT) {  // packed trees only: more than TREE_MAX nodes
        const float fill = slot_of(p, j) < 0 ? 0.f : __builtin_nanf("");
        Out *o = reinterpret_cast<Out *>(p.o) + hv * V;
        for (int64_t i = bos * V + threadIdx.x; i < eos * V; i += 2 * V) o[i / V * p.Hv * V + i % V] = (Out)fill;
        return;
    }
    if constexpr (NT == 4) {
        if (n > 48) return tree<In, Out, K, V, 4>(p, smem, j, hv, bos, (int)n);
        if (n > 32) return tree<In, Out, K, V, 3>(p, smem, j, hv, bos, (int)n);
    }
    if constexpr (NT >= 2)
        if (n > 16) return tree<In, Out, K, V, 2>(p, smem, j, hv, bos, (int)n);
    tree<In, Out, K, V, 1>(p, smem, j, hv, bos, (int)n);
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
