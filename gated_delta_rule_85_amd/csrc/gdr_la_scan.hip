// gdr_la_scan: linear attention with a decay for each head, scanned over chunks of 64 tokens.
//
// Per (sequence, v head), with the state S (KD x W, fp32):
//     S_t = e^{g_t} S_{t-1} + in_scale k_t v_t^T,    o_t = out_scale S_t^T q_t.
// A chunk of n tokens that meets the state h, with gam the running sums of its gates:
//     O  = e^{gam_r} Q h + P V,   P = (Q K^T) in_scale e^{gam_r - gam_i} where i <= r,
//     h' = e^{gam_last} h + K^T diag(in_scale e^{gam_last - gam}) V.
//
// A workgroup of NW waves owns 16 NW columns of S for a whole sequence (or segment), 16 a wave, in
// registers; columns are independent, so the waves share only what is made of K and Q alone: the ten
// 16 x 16 tiles of P on and below the diagonal, through LDS.  A chunk's P V is taken with the next
// chunk's work, so that one barrier a chunk orders everything: in turn c a wave stores O of chunk
// c - 1 with its P V, makes its tiles of P of chunk c and its columns of Q h, then h', while K, Q, V
// and the gates of chunk c + 1 are copied global -> LDS (bf16: two buffers).  NW is 8 (128 columns:
// half of the tiles of P a column) for bf16 inputs where that leaves a workgroup for every compute
// unit, else 4.  Where the LDS has room (KS 2: bf16 in and out, no dots), 8 waves take these 64 columns
// too, in pairs with half of the rows of S each, so that a SIMD has two waves: a wave's part of Q h
// for its partner's rows of the chunk goes through LDS (16 KB a chunk), and P V is split by those
// rows.  Two prompts of 8 heads of 64 columns, 2048 tokens: 72 us in place of 89; 4 x 4096 tokens of
// 32 heads of 128: 167 in place of 185.
//
// Bound by the issue of instructions and the chain of a chunk's steps, at two waves a SIMD: some wave issues in
// 62% of the SIMDs' cycles (pairs: 77%), matrix units are busy in 37% (30%), the LDS in 34% (37%).
// 8 x 4096 tokens of 64 heads, bf16: 528 us, 0.8 PFLOP/s of matrix instructions; the backward's scans
// with their dots and three pieces 740 and 725 us, dk with two 565.
//
// rev: row r of a chunk is its r-th token from the end, and a row's gate is the next token's, so
// that the same code scans from the last token to the first.
//
// Precision: q, k and v in bf16 are exact operands.  h, P and the decayed V are fp32 and enter the
// bf16 matrix instructions in pieces of 8 bits each, x = hi + mid + lo to 2^-25 or hi + mid to
// 2^-17.  The state always takes three.  A bf16 output, or one that is rounded to bf16 after its sum
// over heads, takes two of h and P: its own rounding is 2^-9.  An fp32 output, and the sums that gate gradients are differences of, take three.  fp32
// inputs use the fp32 matrix instruction.
#include "gdr_la.hpp"

namespace gdr {
namespace {


// A gate below this empties the state like this one: e^-104 is 0 in fp32.  (Sums of gates stay
// finite, and -inf may be given.)
constexpr float LOWEST_GATE = -104.f;

// memory that is not LDS: a pointer out of a parameter block would be taken for either
template <typename T> using Glb = __attribute__((address_space(1))) T;
template <typename T> __device__ __forceinline__ Glb<T> *glb(T *p) { return (Glb<T> *)p; }

// Wave-wide copies of 64 x 16 (or 4) bytes global -> LDS, lane l's to 16 l (4 l) past `to`.  As
// instructions of their own: before any read of LDS the compiler waits for every copy that it knows to
// be in flight, whichever buffer is read, and with it for the latency of memory in every chunk.
// Nothing else here uses m0, which the compiler reserves: it holds no value there, and warns of a
// clobber.  wait_copies() and a barrier come before what is copied is read.
__device__ __forceinline__ void copy16(const char *base, uint32_t off, const char *to) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2"
                 :
                 : "s"(__builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)to)), "v"(off), "s"(base)
                 : "memory");
}
__device__ __forceinline__ void copy4(const char *base, uint32_t off, const char *to) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, %2"
                 :
                 : "s"(__builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)to)), "v"(off), "s"(base)
                 : "memory");
}
// until no more than the last N instructions that touch memory are under way: they end in order, and any
// others than copies among them make the wait longer, never shorter
template <int N = 0> __device__ __forceinline__ void wait_copies() { asm volatile("s_waitcnt vmcnt(%0)" : : "n"(N) : "memory"); }

// ------------------------------------------------------- operands in pieces
template <typename In, int NP> struct Pieces {
    bf16x8 p[NP];
};
template <int NP> struct Pieces<float, NP> {
    OpF x;
};

__device__ __forceinline__ f32x4 widen(bf16x4 x) {
    typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
    const u32x2 u = __builtin_bit_cast(u32x2, x);
    return f32x4{__builtin_bit_cast(float, u[0] << 16), __builtin_bit_cast(float, u[0] & 0xffff0000u),
                 __builtin_bit_cast(float, u[1] << 16), __builtin_bit_cast(float, u[1] & 0xffff0000u)};
}
__device__ __forceinline__ bf16x4 narrow(f32x4 x) {
    typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
    const uint32_t a = __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{x[0], x[1]}, bf16x2));
    const uint32_t b = __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{x[2], x[3]}, bf16x2));
    return __builtin_bit_cast(bf16x4, (u32x2{a, b}));
}
template <int NP> __device__ __forceinline__ void pieces4(f32x4 x, bf16x4 (&out)[NP]) {
#pragma unroll
    for (int i = 0; i < NP; ++i) {
        out[i] = narrow(x);
        if (i + 1 < NP) x -= widen(out[i]);
    }
}
template <typename In, int NP> __device__ __forceinline__ Pieces<In, NP> pieces8(f32x4 a, f32x4 b) {
    Pieces<In, NP> r;
    if constexpr (sizeof(In) == 4) {
        r.x = OpF{a, b};
    } else {
        bf16x4 x[NP], y[NP];
        pieces4<NP>(a, x);
        pieces4<NP>(b, y);
#pragma unroll
        for (int i = 0; i < NP; ++i) r.p[i] = cat(x[i], y[i]);
    }
    return r;
}
// c[i] += a b[i] (a[i] b): a piece of all of them before the next, small pieces first, so that a product
// does not wait for the one before it
template <int N, int NP> __device__ __forceinline__ void mma_each(f32x4 *c, const Pieces<bf16, NP> &a, const OpX (&b)[N]) {
#pragma unroll
    for (int k = NP - 1; k >= 0; --k)
#pragma unroll
        for (int i = 0; i < N; ++i) c[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.p[k], cat(b[i].b0, b[i].b1), c[i], 0, 0, 0);
}
template <int N, int NP> __device__ __forceinline__ void mma_each(f32x4 *c, const OpX (&a)[N], const Pieces<bf16, NP> &b) {
#pragma unroll
    for (int k = NP - 1; k >= 0; --k)
#pragma unroll
        for (int i = 0; i < N; ++i) c[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(cat(a[i].b0, a[i].b1), b.p[k], c[i], 0, 0, 0);
}
template <int N, int NP> __device__ __forceinline__ void mma_each(f32x4 *c, const Pieces<float, NP> &a, const OpF (&b)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) c[i] = mma(c[i], a.x, b[i]);
}
template <int N, int NP> __device__ __forceinline__ void mma_each(f32x4 *c, const OpF (&a)[N], const Pieces<float, NP> &b) {
#pragma unroll
    for (int i = 0; i < N; ++i) c[i] = mma(c[i], a[i], b.x);
}
// c[i] += a b[i], b in pieces
template <int N, int NP> __device__ __forceinline__ void mma_pieces(f32x4 *c, const OpX &a, const Pieces<bf16, NP> *b) {
#pragma unroll
    for (int k = NP - 1; k >= 0; --k)
#pragma unroll
        for (int i = 0; i < N; ++i) c[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(cat(a.b0, a.b1), b[i].p[k], c[i], 0, 0, 0);
}
template <int N, int NP> __device__ __forceinline__ void mma_pieces(f32x4 *c, const OpF &a, const Pieces<float, NP> *b) {
#pragma unroll
    for (int i = 0; i < N; ++i) c[i] = mma(c[i], a, b[i].x);
}

// ------------------------------------------------------------ LDS layout
template <typename In, int KD, int NP, int NW, int KS, bool OUT> struct Lay {
    static constexpr bool BF = sizeof(In) == 2;
    // buffers: as many as the two workgroups of a compute unit without output, or the one with it, have room for
    static constexpr int ES = sizeof(In), NB = !BF ? 1 : OUT ? 2 : 3, BW = 16 * NW / KS;
    static constexpr int KROW = KD * ES, VROW = BW * ES, PROW = CH * ES;
    static constexpr int KT = CH * KROW, VT = CH * VROW;
    static constexpr int OFF_K = 0, OFF_V = KT, OFF_Q = KT + VT, BUF = KT + VT + (OUT ? KT : 0);
    static constexpr int PPLANE = CH * PROW, PT = (BF ? NP : 1) * PPLANE;  // planes of P
    static constexpr int OFF_P = NB * BUF;                           // P of two chunks
    static constexpr int OFF_S = OFF_P + (OUT ? 2 * PT : 0);         // dots of two chunks: [wave][token]
    static constexpr int OFF_T = OFF_S + (OUT ? 2 * NW * CH * 4 : 0);  // gate tables of two chunks (without output: of each wave)
    static constexpr int GT = (OUT ? 8 : 3) * CH;                    // floats of one
    static constexpr int OFF_G = OFF_T + (OUT ? 2 : NW) * GT * 4;    // gates of four chunks
    static constexpr int OFF_X = OFF_G + 4 * CH * 4;                 // of two chunks: what a wave adds to its partner's rows
    static constexpr int BYTES = OFF_X + (KS > 1 ? 2 * NW * 2048 : 0);
    static_assert(BYTES <= 160 * 1024, "LDS of a compute unit");
    using SK = Swz<KROW, KeyKQ>;
    using SV = Swz<VROW, typename std::conditional<VROW == 128, KeyVP, KeyKQ>::type>;
    using SP = Swz<PROW, typename std::conditional<BF, KeyP, KeyVP>::type>;
};
// A chunk's table of gates: decays from its start to a row (as the output's factor, too) and from a
// row to its end; and base-2 logarithms of the decay between a key and a row.  Every logarithm is a
// sum of gates that lie between the two alone, never a difference of longer sums: one gate that
// empties the state is -150 here, and a difference of sums past it would keep their rounding, 2^-17.
// Key and row in different tiles of 16: the row's part, from the start of its tile, and the key's,
// to the end of its tile and of d - 1 tiles more for a row tile d tiles on.  In the same tile the
// wave adds the gates itself (between(); a prompt of 4096 tokens of 32 heads, unsplit, in 141 us, with
// tables of such sums in 149).
enum { G_START = 0, G_OUT = CH, G_END = 2 * CH, G_ROW = 3 * CH, G_GATE = 4 * CH, G_KEY = 5 * CH };
__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// one row's gate per lane (0 past the chunk's n rows and before its sequence's first gate) -> the table;
// rows past n add nothing.  PAIRS: with the decays between keys and rows
template <bool PAIRS> __device__ __forceinline__ void gate_table(float gate, int n, float in_scale, float out_scale, float *t) {
    const int l = lane_id(), tile = l >> 4;
    gate = (gate < LOWEST_GATE ? LOWEST_GATE : gate) * 1.4426950408889634f;  // log2 e
    float x = gate;
    x += dpp_mov<0x111>(x);  // row_shr 1, 2, 4, 8: running sums within 16 lanes
    x += dpp_mov<0x112>(x);
    x += dpp_mov<0x114>(x);
    x += dpp_mov<0x118>(x);
    float rest = dpp_mov<0x101>(gate);  // row_shl: of the lanes after this one, to the end of the tile
    rest += dpp_mov<0x101>(rest);
    rest += dpp_mov<0x102>(rest);
    rest += dpp_mov<0x104>(rest);
    rest += dpp_mov<0x108>(rest);
    auto total = [&](int i) { return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, x), i)); };
    const float t0 = total(15), t1 = total(31), t2 = total(47), t3 = total(63);
    const float before = tile == 0 ? 0.f : tile == 1 ? t0 : tile == 2 ? t0 + t1 : t0 + t1 + t2;
    const float next = tile == 0 ? t1 : tile == 1 ? t2 : t3, next2 = tile == 0 ? t2 : t3;
    const float after = tile == 0 ? t1 + t2 + t3 : tile == 1 ? t2 + t3 : tile == 2 ? t3 : 0.f;
    const float start = exp2_fast(before + x);
    t[G_START + l] = start;
    t[G_OUT + l] = out_scale * start;
    t[G_END + l] = l < n ? in_scale * exp2_fast(rest + after) : 0.f;
    if (!PAIRS) return;
    t[G_ROW + l] = x;
    t[G_GATE + l] = gate;
    t[G_KEY + l] = rest;
    t[G_KEY + CH + l] = rest + next;
    t[G_KEY + 2 * CH + l] = rest + (next + next2);
}

// Sums of a tile's gates from after key 4g + i to row n16, where i is not past it: of the lane's own
// gate, over the 16 lanes with the same g, and of those of its keys
__device__ __forceinline__ f32x4 between(float row, const f32x4 &keys) {
    const int after = ln16() - 4 * lg4();  // of key 4g
    float x = after > 3 ? row : 0.f;
    x += dpp_mov<0x111>(x);
    x += dpp_mov<0x112>(x);
    x += dpp_mov<0x114>(x);
    x += dpp_mov<0x118>(x);
    const float x2 = x + (after > 2 ? keys[3] : 0.f), x1 = x2 + (after > 1 ? keys[2] : 0.f);
    return f32x4{x1 + (after > 0 ? keys[1] : 0.f), x1, x2, x};
}

// Sums of four values over the lanes with the same l & 15: of value [0, 2, 1, 3][l >> 4]
__device__ __forceinline__ float sum_rows(f32x4 x) {
    auto add = [](auto r) {
        const uint32_t a = r[0], b = r[1];
        return __builtin_bit_cast(float, a) + __builtin_bit_cast(float, b);
    };
    auto bits = [](float x) { return __builtin_bit_cast(uint32_t, x); };
    const float a = add(__builtin_amdgcn_permlane32_swap(bits(x[0]), bits(x[1]), false, false));
    const float b = add(__builtin_amdgcn_permlane32_swap(bits(x[2]), bits(x[3]), false, false));
    return add(__builtin_amdgcn_permlane16_swap(bits(a), bits(b), false, false));
}

// ------------------------------------------------------- a workgroup's part
// Out: void for the end states of segments alone; DOTS: LaJob's sums with e
template <typename In, typename Out, int KD, int NP, int NW, int KS, bool DOTS> struct Scan {
    static constexpr bool OUT = !std::is_void<Out>::value;
    using Y = Lay<In, KD, NP, NW, KS, OUT>;
    using SK = typename Y::SK;
    using SV = typename Y::SV;
    using SP = typename Y::SP;
    using X = typename Ops<In>::X;
    static constexpr int ES = Y::ES, BW = Y::BW, RT = KD / 16 / KS, U = KD / 32;  // tiles of 16 rows of h on a wave; of 32 rows of all of it
    static_assert(KS == 1 || (KS == 2 && OUT && !DOTS), "");

    const LaParams &p;
    const LaJob &J;
    char *const lds;
    int cb, hv, j, m, len, nc, n_it, c_first, first_place, before_border;
    int64_t bos;
    bool rev, starts, ends;
    int l, n16, g, w;
    // the wave's columns 16 ct .. and rows row0 .. of h, the part-th of KS
    __device__ __forceinline__ int ct() const { return KS == 1 ? w : w % (NW / KS); }
    __device__ __forceinline__ int part() const { return KS == 1 ? 0 : w / (NW / KS); }
    __device__ __forceinline__ int row0() const { return part() * (KD / KS); }

    __device__ __forceinline__ Scan(const LaParams &p_, int job, char *lds_) : p(p_), J(p_.job[job]), lds(lds_) {}

    // false: nothing to do
    __device__ __forceinline__ bool place(int item) {
        j = item, m = 0;
        if (p.split && !la_place(p.s, item, j, m)) return false;
        int64_t eos;
        la_bounds(p.s, j, bos, eos);
        rev = J.rev;
        len = (int)(eos - bos), nc = (len + CH - 1) / CH;
        first_place = la_first(p.s, bos, j, (int64_t)p.s.seg_chunks * CH);
        before_border = la_before(p.s, bos, j, (int64_t)p.s.seg_chunks * CH);
        const int n_seg = p.split ? max(1, (nc + p.s.seg_chunks - 1) / p.s.seg_chunks) : 1;
        const int c_lo = p.split ? m * p.s.seg_chunks : 0, c_hi = p.split ? min(nc, c_lo + p.s.seg_chunks) : nc;
        n_it = c_hi - c_lo, c_first = rev ? c_hi - 1 : c_lo;
        starts = m == (rev ? n_seg - 1 : 0), ends = m == (rev ? 0 : n_seg - 1);
        l = lane_id(), n16 = ln16(), g = lg4();
        w = __builtin_amdgcn_readfirstlane(wave_id());
        return true;
    }
    __device__ __forceinline__ int chunk_of(int it) const { return rev ? c_first - it : c_first + it; }
    __device__ __forceinline__ int rows_of(int c) const { return min(CH, len - c * CH); }
    // row r of a chunk of n rows -> its token counted from the chunk's first
    __device__ __forceinline__ int token_of(int r, int n) const { return rev ? n - 1 - r : r; }
    // element offset of the sequence's first token in a tensor
    __device__ __forceinline__ int64_t first_row(int64_t row, int64_t batch) const { return p.s.cu ? bos * row : (int64_t)j * batch; }

    // ----------------------------------------------------------------- states
    // h[t][i]: row row0 + slot_base(t, g) + i, column 16 ct + n16 of the block
    __device__ __forceinline__ void load_state(const float *s, f32x4 (&h)[RT]) const {
        const int col = cb * BW + 16 * ct() + n16;
#pragma unroll
        for (int t = 0; t < RT; ++t) {
            const int r = row0() + slot_base(t, g);
            if (J.trans) {
                h[t] = *glb(reinterpret_cast<const f32x4 *>(s + (int64_t)col * KD + r));
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) h[t][i] = glb(s)[(r + i) * J.W + col];
            }
        }
    }
    __device__ __forceinline__ void store_state(float *s, const f32x4 (&h)[RT], float f) const {
        const int col = cb * BW + 16 * ct() + n16;
#pragma unroll
        for (int t = 0; t < RT; ++t) {
            const int r = row0() + slot_base(t, g);
            if (J.trans) {
                *glb(reinterpret_cast<f32x4 *>(s + (int64_t)col * KD + r)) = f * h[t];
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) glb(s)[(r + i) * J.W + col] = f * h[t][i];
            }
        }
    }
    __device__ __forceinline__ float *at_place(float *s, int at) const { return s + ((int64_t)at * p.s.Hv + hv) * KD * J.W; }
    __device__ __forceinline__ int64_t unit() const { return (int64_t)j * p.s.Hv + hv; }
    __device__ __forceinline__ void start_state(f32x4 (&h)[RT]) const {
        if (starts ? J.init != nullptr : OUT) {
            load_state(starts ? J.init + unit() * KD * J.W : at_place(J.border, before_border + (rev ? m + 1 : m)), h);
        } else {
#pragma unroll
            for (int t = 0; t < RT; ++t) h[t] = zero4();
        }
    }
    __device__ __forceinline__ void end_state(const f32x4 (&h)[RT]) const {
        if (ends && J.fin) {
            float f = 1.f;
            if (rev && len > 0) f = fast_exp(p.s.g[bos * p.s.g_tok + hv]);
            store_state(J.fin + unit() * KD * J.W, h, f);
        }
        if constexpr (DOTS)
            if (ends && J.with) {
                const float *s = J.with + unit() * KD * J.W + (int64_t)(cb * BW + 16 * ct() + n16) * KD;
                f32x4 d = zero4(), v = zero4();
#pragma unroll
                for (int t = 0; t < RT; ++t) {
                    const f32x4 z = h[t] * *glb(reinterpret_cast<const f32x4 *>(s + row0() + slot_base(t, g)));
                    d += z, v += z * z;
                }
                double2 x = {(double)((d[0] + d[1]) + (d[2] + d[3])), (double)((v[0] + v[1]) + (v[2] + v[3]))};
#pragma unroll
                for (int i = 32; i; i >>= 1) x.x += __shfl_xor(x.x, i), x.y += __shfl_xor(x.y, i);
                if (l == 0) J.last[unit() * (J.W / 16) + cb * (BW / 16) + ct()] = x;
            }
    }

    // ----------------------------------------------------------------- copies
    // Pieces of 1 KB in turn on the waves, and the gates.  The offsets of a lane's rows and 16-byte
    // columns are the same in every whole chunk; rows past the end of a shorter one repeat its last row.
    static constexpr int NK = Y::KT / 1024 / NW, NV = Y::VT / 1024 / NW;
    static_assert(NK * 1024 * NW == Y::KT && NV * 1024 * NW == Y::VT, "pieces spread over the waves");
    struct Copies {
        const char *k, *q, *v;    // first row of the chunk to copy next
        int64_t k_step, q_step, v_step;
        uint32_t ko[NK], qo[OUT ? NK : 1], vo[NV];
        int at;                   // that chunk's first token
    };
    template <typename S> __device__ __forceinline__ uint32_t copy_offset(int i, uint32_t row, int n) const {
        constexpr int ROWB = S::CPR * 16;
        const int b = (NW * i + w) * 1024 + 16 * l, r = b / ROWB, pc = (b % ROWB) / 16;
        return (uint32_t)token_of(min(r, n - 1), n) * row + 16 * S::chunk(r, pc);
    }
    __device__ __forceinline__ Copies copies() const {
        Copies x;
        x.at = c_first * CH;
        auto from = [&](const void *t, int64_t row, int64_t batch, int head, int64_t &step) {
            step = (rev ? -CH : CH) * row * ES;
            return reinterpret_cast<const char *>(t) + (first_row(row, batch) + x.at * row + head) * ES;
        };
        x.k = from(J.k, J.k_row, J.k_batch, (hv / J.k_div) * KD, x.k_step);
        x.v = from(J.v, J.v_row, J.v_batch, (hv / J.v_div) * J.W + cb * BW, x.v_step);
        x.q = OUT ? from(J.q, J.q_row, J.q_batch, (hv / J.q_div) * KD, x.q_step) : nullptr;
#pragma unroll
        for (int i = 0; i < NK; ++i) {
            x.ko[i] = copy_offset<SK>(i, (uint32_t)(J.k_row * ES), CH);
            if constexpr (OUT) x.qo[i] = copy_offset<SK>(i, (uint32_t)(J.q_row * ES), CH);
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) x.vo[i] = copy_offset<SV>(i, (uint32_t)(J.v_row * ES), CH);
        return x;
    }
    // the next chunk -> buffer buf
    __device__ __forceinline__ void issue(Copies &x, int buf) const {
        char *b = buffer(buf);
        const int n = min(CH, len - x.at);
        if (__builtin_expect(n == CH, 1)) {
#pragma unroll
            for (int i = 0; i < NK; ++i) {
                copy16(x.k, x.ko[i], b + Y::OFF_K + (NW * i + w) * 1024);
                if constexpr (OUT) copy16(x.q, x.qo[i], b + Y::OFF_Q + (NW * i + w) * 1024);
            }
#pragma unroll
            for (int i = 0; i < NV; ++i) copy16(x.v, x.vo[i], b + Y::OFF_V + (NW * i + w) * 1024);
        } else {
#pragma unroll 1
            for (int i = 0; i < NK; ++i) {
                copy16(x.k, copy_offset<SK>(i, (uint32_t)(J.k_row * ES), n), b + Y::OFF_K + (NW * i + w) * 1024);
                if constexpr (OUT) copy16(x.q, copy_offset<SK>(i, (uint32_t)(J.q_row * ES), n), b + Y::OFF_Q + (NW * i + w) * 1024);
            }
#pragma unroll 1
            for (int i = 0; i < NV; ++i) copy16(x.v, copy_offset<SV>(i, (uint32_t)(J.v_row * ES), n), b + Y::OFF_V + (NW * i + w) * 1024);
        }
        x.k += x.k_step, x.v += x.v_step, x.at += rev ? -CH : CH;
        if constexpr (OUT) x.q += x.q_step;
    }
    __device__ __forceinline__ char *buffer(int buf) const { return lds + (Y::NB > 1 ? buf * Y::BUF : 0); }

    // Gates: copied two chunks ahead into one of four places, made into a table one chunk ahead.  One
    // wave does both.
    __device__ __forceinline__ void issue_gates(int it) const {
        const int c = chunk_of(it), n = rows_of(c), t = c * CH + min(max(rev ? n - l : l, 0), min(CH, len - c * CH - 1));
        const char *from = reinterpret_cast<const char *>(p.s.g + (bos + c * (int64_t)CH) * p.s.g_tok + hv);
        copy4(from, (uint32_t)(t - c * CH) * (uint32_t)(4 * p.s.g_tok), lds + Y::OFF_G + (it & 3) * CH * 4);
    }
    __device__ __forceinline__ void make_table(int it, float *to) const {
        const int c = chunk_of(it), n = rows_of(c), t = c * CH + (rev ? n - l : l);
        const float x = reinterpret_cast<const float *>(lds + Y::OFF_G)[(it & 3) * CH + l];
        gate_table<OUT>(l < n && t < len ? x : 0.f, n, J.in_scale, OUT ? J.out_scale : 1.f, to);
    }
    __device__ __forceinline__ float *table(int buf) const { return reinterpret_cast<float *>(lds + Y::OFF_T) + buf * Y::GT; }

    // --------------------------------------------------------------- products
    // The reads of LDS that a product needs, and the product, apart: run() reads for one step during
    // the step before, and stage() keeps the compiler from moving the reads to where they are used.
    static __device__ __forceinline__ void stage() { __builtin_amdgcn_sched_barrier(0); }

    // V^T of this wave's columns and keys 32 ip ..
    __device__ __forceinline__ X values(const char *b, int ip) const { return kt8<In, SV>(b + Y::OFF_V, 32 * ip, 16 * ct(), 4); }
    // those, decayed to the chunk's end
    struct Ends {
        f32x4 e[2][2];
    };
    __device__ __forceinline__ Ends ends_of(const float *gt) const {
        Ends x;
#pragma unroll
        for (int ip = 0; ip < 2; ++ip)
#pragma unroll
            for (int i = 0; i < 2; ++i) x.e[ip][i] = *reinterpret_cast<const f32x4 *>(gt + G_END + 32 * ip + 8 * g + 4 * i);
        return x;
    }
    __device__ __forceinline__ Pieces<In, 3> decayed(const X &v, const f32x4 (&e)[2]) const {
        if constexpr (Y::BF)
            return pieces8<In, 3>(widen(v.b0) * e[0], widen(v.b1) * e[1]);
        else
            return pieces8<In, 3>(v.b0 * e[0], v.b1 * e[1]);
    }
    // K^T of tiles T .. T + N - 1, keys 32 ip ..
    static constexpr int N4 = !Y::BF ? 2 : RT < 4 ? RT : 4;  // (fp32: registers)
    struct Keys {
        X k[N4];
    };
    __device__ __forceinline__ Keys keys(const char *b, int ip, int first) const {
        Keys x;
#pragma unroll
        for (int i = 0; i < N4; ++i) {
            const int t = first + i;
            x.k[i] = kt8<In, SK>(b + Y::OFF_K, 32 * ip, row0() + 32 * (t >> 1) + 4 * (t & 1), 8);
        }
        return x;
    }
    __device__ __forceinline__ void add_keys(const Keys &k, const Pieces<In, 3> &d, int first, f32x4 (&h)[RT]) const {
        mma_each<N4>(h + first, k.k, d);
    }
    // h to the chunk's end; the first keys have been read
    __device__ __forceinline__ void add_chunk(const char *b, const float *gt, const X (&v)[2], const Ends &e, Keys k, f32x4 (&h)[RT]) const {
        const float all = gt[G_START + CH - 1];
        const Pieces<In, 3> d0 = decayed(v[0], e.e[0]);
#pragma unroll
        for (int t = 0; t < RT; ++t) h[t] *= all;
        Pieces<In, 3> d1;
#pragma unroll
        for (int i = 0; i < 2 * RT / N4; ++i) {
            const int ip = i / (RT / N4), first = i % (RT / N4) * N4, j = i + 1;
            stage();
            Keys next;
            if (j < 2 * RT / N4) next = keys(b, j / (RT / N4), j % (RT / N4) * N4);
            add_keys(k, ip ? d1 : d0, first, h);
            if (i == 0) d1 = decayed(v[1], e.e[1]);
            k = next;
        }
        stage();
    }
    __device__ __forceinline__ X query(const char *b, int rt, int u) const {
        return frag8<In, SK>(b + Y::OFF_Q, 16 * rt + n16, (32 * u + 8 * g) * ES);
    }
    __device__ __forceinline__ X key(const char *b, int kt, int u) const {
        return frag8<In, SK>(b + Y::OFF_K, 16 * kt + n16, (32 * u + 8 * g) * ES);
    }
    // N tiles of P of one row tile
    template <int N> struct Scores {
        X k[N][U], q[U];
        f32x4 key[N];
        float row[N];
    };
    template <int N> __device__ __forceinline__ Scores<N> score_operands(const char *b, const float *gt, int rt, int kt) const {
        Scores<N> x;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            x.q[u] = query(b, rt, u);
#pragma unroll
            for (int i = 0; i < N; ++i) x.k[i][u] = key(b, kt + i, u);
        }
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int d = rt - kt - i;
            x.key[i] = *reinterpret_cast<const f32x4 *>(gt + (d ? G_KEY + (d - 1) * CH : G_GATE) + 16 * (kt + i) + 4 * g);
            x.row[i] = gt[(d ? G_ROW : G_GATE) + 16 * rt + n16];
        }
        return x;
    }
    template <int N> __device__ __forceinline__ void score(const Scores<N> &x, char *P, int rt, int kt) const {
        f32x4 s[N];
#pragma unroll
        for (int i = 0; i < N; ++i) s[i] = zero4();
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < N; ++i) s[i] = mma(s[i], x.k[i][u], x.q[u]);
        const float scale = J.in_scale * J.out_scale;
#pragma unroll
        for (int i = 0; i < N; ++i) {  // s[i][k]: row 16 rt + n16, key 16 (kt + i) + 4g + k
            const bool same = rt == kt + i;
            f32x4 log;
            if (same)
                log = between(x.row[i], x.key[i]);
            else
                log = x.row[i] + x.key[i];
#pragma unroll
            for (int k = 0; k < 4; ++k) s[i][k] = !same || 4 * g + k <= n16 ? s[i][k] * (scale * exp2_fast(log[k])) : 0.f;
            char *to = P + SP::off(16 * rt + n16, (16 * (kt + i) + 4 * g) * ES);
            if constexpr (Y::BF) {
                bf16x4 y[NP];
                pieces4<NP>(s[i], y);
#pragma unroll
                for (int k = 0; k < NP; ++k) *reinterpret_cast<bf16x4 *>(to + k * Y::PPLANE) = y[k];
            } else {
                *reinterpret_cast<f32x4 *>(to) = s[i];
            }
        }
    }
    // P of N of this wave's own row tiles from the first on, keys 32 ip ..
    // a wave's order of the chunk's row tiles: every KS-th is its own, the one after its partner's
    __device__ __forceinline__ int row_tile(int i) const { return KS == 1 ? i : i ^ part(); }
    template <int N> struct Weights {
        Pieces<In, NP> p[N];
    };
    template <int N> __device__ __forceinline__ Weights<N> weights(const char *P, int first, int ip) const {
        Weights<N> x;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int row = 16 * row_tile(KS * (first + i)) + n16, off = SP::off(row, (32 * ip + 8 * g) * ES);
            if constexpr (Y::BF) {
#pragma unroll
                for (int k = 0; k < NP; ++k) x.p[i].p[k] = *reinterpret_cast<const bf16x8 *>(P + k * Y::PPLANE + off);
            } else {
                x.p[i].x.b0 = *reinterpret_cast<const f32x4 *>(P + off);
                x.p[i].x.b1 = *reinterpret_cast<const f32x4 *>(P + SP::off(row, (32 * ip + 8 * g) * ES + 16));
            }
        }
        return x;
    }

    // --------------------------------------------------------------- the waves
    // Two chunks a turn, so that a buffer's addresses are the same in every turn
    template <typename F> __device__ __forceinline__ void each_chunk(F step) const {
        for (int it = 0; it < n_it; it += 2) {
            step(it, std::integral_constant<int, 0>{});
            if (it + 1 < n_it) step(it + 1, std::integral_constant<int, 1>{});
        }
    }
    __device__ __forceinline__ void first_copies(Copies &x, bool with_gates) const {
        if (n_it > 0) {
            issue(x, 0);
            if (with_gates) {
                issue_gates(0);
                if (n_it > 1) issue_gates(1);
                wait_copies();
                make_table(0, table(0));  // (this wave's own copy)
            }
        }
        wait_copies();
        lds_barrier();
    }

    __device__ __forceinline__ void run() {
        Copies from = copies();
        f32x4 h[RT];
        start_state(h);
        int to_border = !J.border || p.split ? -1 : rev ? c_first % p.s.seg_chunks + 1 : p.s.seg_chunks;  // chunks
        // the tiles of P right of the diagonal that a 32-deep product reads: zero, never written
        constexpr int per = 16 * 16 * 2;  // elements of a plane
        for (int i = threadIdx.x; i < 2 * (Y::PT / Y::PPLANE) * per; i += 64 * NW) {
            const int e = i % per, t = e >> 8, r = 32 * t + ((e >> 4) & 15), k = 32 * t + 16 + (e & 15);
            *reinterpret_cast<In *>(lds + Y::OFF_P + (i / per) * Y::PPLANE + SP::off(r, k * ES)) = In(0.f);
        }
        typedef In in4 __attribute__((ext_vector_type(4)));
        typedef Out out4 __attribute__((ext_vector_type(4)));
        // a row's place: token 16 r + n16 of the chunk, columns 4g .. of this wave's.  Offsets within a
        // whole chunk; a shorter one's rows lie that much lower where rows run backwards
        const int64_t orow = (int64_t)p.s.Hv * J.W, at = c_first * (int64_t)CH;
        const int in_block = cb * BW + 16 * ct() + 4 * g;
        Out *o0 = reinterpret_cast<Out *>(J.o) + (bos + at) * orow + (int64_t)hv * J.W + in_block;
        const int64_t o_step = (rev ? -CH : CH) * orow;
        const In *e0 = nullptr;
        float *d0 = nullptr;
        uint32_t oo[4], eo[4];
#pragma unroll
        for (int r = 0; r < 4; r += KS) {
            const int tok = token_of(16 * row_tile(r) + n16, CH);
            oo[r] = (uint32_t)tok * (uint32_t)orow;
            if constexpr (DOTS) eo[r] = (uint32_t)tok * (uint32_t)J.e_row;
        }
        if constexpr (DOTS) {
            e0 = reinterpret_cast<const In *>(J.e) + first_row(J.e_row, J.e_batch) + at * J.e_row + (hv / J.e_div) * J.W + in_block;
            d0 = J.dots + ((int64_t)cb * p.s.Hv + hv) * p.tokens + bos;
        }
        auto dots_at = [&](int buf) { return reinterpret_cast<float *>(lds + Y::OFF_S) + buf * NW * CH; };
        auto store_dots = [&](int it, int buf) {  // one wave, a row per lane
            const int c = chunk_of(it), n = rows_of(c);
            double d = 0.0;  // (gate gradients are what is left of many of these)
#pragma unroll
            for (int i = 0; i < NW; ++i) d += (double)dots_at(buf)[i * CH + l];
            if (l < n) glb(d0)[c * CH + token_of(l, n)] = (float)d;
        };
        // of the chunk before: its Q h, V and part of e
        f32x4 o[4] = {zero4(), zero4(), zero4(), zero4()};
        X v[2];
        v[0] = v[1] = X{};
        in4 e[4];
        auto place_of_scores = [&](int buf) { return lds + Y::OFF_P + buf * Y::PT; };
        // + P V
        constexpr int OT = 4 / KS;  // this wave's own row tiles
        auto add_to = [&](auto first, const X &y, const auto &x) {
            if constexpr (KS == 1) {
                mma_pieces<OT - first>(o + first, y, x.p);
            } else {
                f32x4 z[OT - first];
#pragma unroll
                for (int i = first; i < OT; ++i) z[i - first] = o[KS * i];
                mma_pieces<OT - first>(z, y, x.p);
#pragma unroll
                for (int i = first; i < OT; ++i) o[KS * i] = z[i - first];
            }
        };
        auto add_first = [&](const Weights<OT> &x) { add_to(std::integral_constant<int, 0>{}, v[0], x); };  // keys 0 .. 31 of all rows
        auto add_rest = [&](const Weights<OT / 2> &x) { add_to(std::integral_constant<int, OT / 2>{}, v[1], x); };  // the others
        // the partner's rows, of this wave's part of Q h, to the partner, and back
        auto exchange = [&](int buf, int wave) { return reinterpret_cast<f32x4 *>(lds + Y::OFF_X) + ((buf * NW + wave) * 2) * 64 + l; };
        auto give = [&](int buf) {
            if constexpr (KS > 1) exchange(buf, w)[0] = o[1], exchange(buf, w)[64] = o[3];
        };
        auto take = [&](int buf) {
            if constexpr (KS > 1) o[0] += exchange(buf, w ^ (NW / 2))[0], o[2] += exchange(buf, w ^ (NW / 2))[64];
        };
        auto finish = [&](int it, int buf) {  // chunk `it`, its dots in place buf
            const int n = rows_of(chunk_of(it));
            if constexpr (DOTS) {
                f32x4 d;
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    d[r] = o[r][0] * to_f32(e[r][0]);
#pragma unroll
                    for (int i = 1; i < 4; ++i) d[r] = fmaf(o[r][i], to_f32(e[r][i]), d[r]);
                }
                const int tile = (l >> 5 & 1) | (l >> 3 & 2);
                dots_at(buf)[w * CH + 16 * tile + n16] = sum_rows(d);
            }
            Out *oc = o0 + (rev && n < CH ? (n - CH) * orow : 0);
#pragma unroll
            for (int r = 0; r < 4; r += KS)
                if (16 * row_tile(r) + n16 < n) *glb(reinterpret_cast<out4 *>(oc + oo[r])) = __builtin_convertvector(o[r], out4);
            o0 += o_step;
        };
        constexpr bool TIGHT = NP == 3 || !Y::BF;  // registers for a step less of P
        // this wave's tiles of P: NT of one row tile and, for two waves (of eight: two without gates to add), one more
        constexpr int NT = NW == 8 ? 1 : 2;
        const int rt = NW == 8 ? (w == 0 || w == 6 ? 1 : w == 2 || w == 4 ? 2 : w == 7 ? 0 : 3) : w == 1 ? 1 : w == 2 ? 2 : 3;
        const int kt = NW == 8 ? (w == 1 || w == 2 ? 2 : w == 3 ? 3 : w == 6 ? 1 : 0) : w == 0 ? 2 : 0;
        const int more_rt = NW == 8 ? (w == 4 ? 2 : w == 5 ? 3 : -1) : w == 2 ? 2 : w == 3 ? 0 : -1;
        const int more_kt = NW == 8 ? 1 : w == 2 ? 2 : 0;
        // the waves that make the gate tables and add up the dots: on SIMDs whose waves have one tile each
        constexpr int GATES = NW == 8 ? 3 : 0, SUMS = NW == 8 ? 2 : 1;
        first_copies(from, w == GATES);
        each_chunk([&](int it, auto B) {
            constexpr int buf = decltype(B)::value;
            const int c = chunk_of(it), n = rows_of(c);
            const char *b = buffer(buf);
            const float *gt = table(buf);
            char *P = place_of_scores(buf);
            if (Y::NB == 2 && it + 1 < n_it) issue(from, buf ^ 1);
            stage();
            // the last chunk's P V (in the first turn of zeros), with the reads for the tiles of P
            const char *last = place_of_scores(buf ^ 1);
            const Weights<OT> p0 = weights<OT>(last, 0, 0);
            Weights<OT / 2> p1;
            if (!TIGHT) p1 = weights<OT / 2>(last, OT / 2, 1);
            if (it > 0) take(buf ^ 1);
            stage();
            if (TIGHT) {
                p1 = weights<OT / 2>(last, OT / 2, 1);
                add_first(p0);
                stage();
            }
            const Scores<NT> sc = score_operands<NT>(b, gt, rt, kt);
            if (!TIGHT) add_first(p0);
            add_rest(p1);
            if (it > 0) finish(it - 1, buf ^ 1);
            if constexpr (DOTS) {
                if (w == SUMS && it > 1) store_dots(it - 2, buf);
                const In *ec = e0 + (rev && n < CH ? (n - CH) * J.e_row : 0);
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    if (16 * r + n16 < n) e[r] = *glb(reinterpret_cast<const in4 *>(ec + eo[r]));
                e0 += (rev ? -CH : CH) * J.e_row;
            }
            stage();
            X q[4];
            if (Y::BF)
#pragma unroll
                for (int r = 0; r < 4; ++r) q[r] = query(b, row_tile(r), part() * (U / KS));
            score<NT>(sc, P, rt, kt);
            stage();
            // (Q h)^T: lane (token n16 of tile r, columns 4g ..)
            float out[4];
            Ends ends_here;
            Keys k0;
#pragma unroll
            for (int r = 0; r < 4; ++r) o[r] = zero4();
#pragma unroll
            for (int u = 0; u < U / KS; ++u) {
                const int at = part() * (U / KS) + u;
                X next[4];
                if (!Y::BF)  // (registers)
#pragma unroll
                    for (int r = 0; r < 4; ++r) q[r] = query(b, row_tile(r), at);
                if (u + 1 < U / KS) {
                    if (Y::BF)
#pragma unroll
                    for (int r = 0; r < 4; ++r) next[r] = query(b, row_tile(r), at + 1);
                } else {
                    v[0] = values(b, 0), v[1] = values(b, 1), ends_here = ends_of(gt), k0 = keys(b, 0, 0);
#pragma unroll
                    for (int r = 0; r < 4; ++r) out[r] = gt[G_OUT + 16 * row_tile(r) + n16];
                }
                const Pieces<In, NP> hp = pieces8<In, NP>(h[2 * u], h[2 * u + 1]);
                mma_each<4>(o, hp, q);
                stage();
                if (Y::BF)
#pragma unroll
                    for (int r = 0; r < 4; ++r) q[r] = next[r];
            }
#pragma unroll
            for (int r = 0; r < 4; ++r) o[r] *= out[r];
            give(buf);
            add_chunk(b, gt, v, ends_here, k0, h);
            if (more_rt >= 0) score<1>(score_operands<1>(b, gt, more_rt, more_kt), P, more_rt, more_kt);
            if (w == GATES) {
                if (it + 1 < n_it) make_table(it + 1, table(buf ^ 1));
                if (it + 2 < n_it) issue_gates(it + 2);
            }
            if (--to_border == 0) {
                to_border = p.s.seg_chunks;
                const int after = rev ? c : c + 1;  // chunks before the border
                if (after > 0 && after < nc) store_state(at_place(J.border, before_border + after / p.s.seg_chunks), h, 1.f);
            }
            wait_copies();
            lds_barrier();
            if (Y::NB == 1 && it + 1 < n_it) {
                issue(from, 0);
                wait_copies();
                lds_barrier();
            }
        });
        if (n_it > 0) {
            const char *last = place_of_scores((n_it - 1) & 1);
            take((n_it - 1) & 1);
            add_first(weights<OT>(last, 0, 0));
            add_rest(weights<OT / 2>(last, OT / 2, 1));
            finish(n_it - 1, (n_it - 1) & 1);
            if constexpr (DOTS) {
                lds_barrier();
                if (w == SUMS && n_it > 1) store_dots(n_it - 2, n_it & 1);
                if (w == SUMS) store_dots(n_it - 1, (n_it - 1) & 1);
            }
        }
        end_state(h);
    }

    // The end state of a segment alone.  Its chunks take less time than memory's latency, so that two
    // (bf16) are copied ahead; every wave copies the gates, so that all have as many copies under way.
    __device__ __forceinline__ void run_segment() {
        constexpr int AHEAD = Y::NB == 3 ? 2 : 1, EACH = NK + NV + 1;
        static_assert(NK * NW * 1024 == Y::KT && NV * NW * 1024 == Y::VT, "as many copies on every wave");
        Copies from = copies();
        f32x4 h[RT];
        start_state(h);
        float whole = 1.f;
        auto fetch = [&](int it, int buf) {
            issue(from, buf);
            issue_gates(it);
        };
#pragma unroll
        for (int i = 0; i < AHEAD; ++i)
            if (i < n_it) fetch(i, i);
        int buf = 0;
        for (int it = 0; it < n_it; ++it) {
            // chunk it landed, the buffer of it - 1 free
            if (AHEAD == 2 && it + 1 < n_it)
                wait_copies<EACH>();
            else
                wait_copies();
            lds_barrier();
            const char *b = buffer(buf);
            const int next = buf == 0 ? AHEAD : buf - 1;  // of chunk it + AHEAD
            if (Y::NB > 1 && it + AHEAD < n_it) fetch(it + AHEAD, next);
            const X v[2] = {values(b, 0), values(b, 1)};
            const Keys k0 = keys(b, 0, 0);
            make_table(it, table(w));  // a table of its own for each wave
            const float *gt = table(w);
            const Ends e = ends_of(gt);
            add_chunk(b, gt, v, e, k0, h);
            whole *= gt[G_START + CH - 1];
            if (Y::NB == 1) {
                lds_barrier();
                if (it + 1 < n_it) fetch(it + 1, 0);
            }
            buf = buf + 1 == Y::NB ? 0 : buf + 1;
        }
        store_state(at_place(J.border, before_border + (rev ? m : m + 1)), h, 1.f);
        if (cb == 0 && threadIdx.x == 0) J.decays[(int64_t)(first_place + m) * p.s.Hv + hv] = whole;
    }
};

template <typename In, typename Out, int KD, int NP, int NW, int KS, bool DOTS>
__global__ __launch_bounds__(64 * NW)
    __attribute__((amdgpu_waves_per_eu(NW / 4, NW / 4))) void gdr_la_scan_kernel(const LaParams p) {
    using S = Scan<In, Out, KD, NP, NW, KS, DOTS>;
    __shared__ __attribute__((aligned(16))) char lds[S::Y::BYTES];
    int id = la_work(blockIdx.x, gridDim.x, p.share);
    const int cb = id % p.n_cb;
    id /= p.n_cb;
    S s(p, id % p.n_jobs, lds);
    id /= p.n_jobs;
    s.cb = cb, s.hv = id % p.s.Hv;
    if (!s.place(id / p.s.Hv)) return;
    s.run();
}
// end states of segments
template <typename In, int KD>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(2))) void gdr_la_states_kernel(const LaParams p) {
    using S = Scan<In, void, KD, 1, 4, 1, false>;
    __shared__ __attribute__((aligned(16))) char lds[S::Y::BYTES];
    int id = la_work(blockIdx.x, gridDim.x, p.share);
    const int cb = id % p.n_cb;
    id /= p.n_cb;
    S s(p, id % p.n_jobs, lds);
    id /= p.n_jobs;
    s.cb = cb, s.hv = id % p.s.Hv;
    if (s.place(id / p.s.Hv) && !s.ends) s.run_segment();  // (a border lies after it)
}

template <typename In, typename Out, int NP, bool DOTS>
hipError_t launch(int KD, const LaParams &p, int items, hipStream_t s) {
    const dim3 grid((uint32_t)items * p.s.Hv * p.n_jobs * p.n_cb);
    if constexpr (sizeof(In) == 2) {  // (fp32: a wave of 8 would not have the registers)
        if (p.job[0].W == 128 * p.n_cb) {
            if (KD == 128)
                launch_k(gdr_la_scan_kernel<In, Out, 128, NP, 8, 1, DOTS>, grid, dim3(512), 0, s, p);
            else
                launch_k(gdr_la_scan_kernel<In, Out, 64, NP, 8, 1, DOTS>, grid, dim3(512), 0, s, p);
            return hipGetLastError();
        }
    }
    constexpr int KS = sizeof(In) == 2 && NP == 2 && !DOTS ? 2 : 1;  // (more pieces of P: LDS)
    if (KD == 128)
        launch_k(gdr_la_scan_kernel<In, Out, 128, NP, 4 * KS, KS, DOTS>, grid, dim3(256 * KS), 0, s, p);
    else
        launch_k(gdr_la_scan_kernel<In, Out, 64, NP, 4 * KS, KS, DOTS>, grid, dim3(256 * KS), 0, s, p);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_la_scan(Dt dt, Dt out, Dt last, int KD, bool dots, const LaParams &p, int items, hipStream_t s) {
    if (dt == Dt::F32) {
        if (out == Dt::F32) return dots ? launch<float, float, 1, true>(KD, p, items, s) : launch<float, float, 1, false>(KD, p, items, s);
        return dots ? launch<float, bf16, 1, true>(KD, p, items, s) : launch<float, bf16, 1, false>(KD, p, items, s);
    }
    if (out == Dt::F32 && last == Dt::BF16 && !dots) return launch<bf16, float, 2, false>(KD, p, items, s);
    if (out == Dt::F32) return dots ? launch<bf16, float, 3, true>(KD, p, items, s) : launch<bf16, float, 3, false>(KD, p, items, s);
    return dots ? launch<bf16, bf16, 3, true>(KD, p, items, s) : launch<bf16, bf16, 2, false>(KD, p, items, s);
}

hipError_t launch_la_states(Dt dt, int KD, const LaParams &p, int items, hipStream_t s) {
    const dim3 grid((uint32_t)items * p.s.Hv * p.n_jobs * p.n_cb);
    if (dt == Dt::F32 && KD == 128)
        launch_k(gdr_la_states_kernel<float, 128>, grid, dim3(256), 0, s, p);
    else if (dt == Dt::F32)
        launch_k(gdr_la_states_kernel<float, 64>, grid, dim3(256), 0, s, p);
    else if (KD == 128)
        launch_k(gdr_la_states_kernel<bf16, 128>, grid, dim3(256), 0, s, p);
    else
        launch_k(gdr_la_states_kernel<bf16, 64>, grid, dim3(256), 0, s, p);
    return hipGetLastError();
}

}  // namespace gdr
