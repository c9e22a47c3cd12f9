// gdr_la_scan: linear attention with a decay for each head, scanned over chunks of 64 tokens.
//
// Per (sequence, v head), with the state S (KD x W, fp32):
//     S_t = e^{g_t} S_{t-1} + in_scale k_t v_t^T,    o_t = out_scale S_t^T q_t.
// A chunk of n tokens that meets the state h, with gam the running sums of its gates:
//     O  = e^{gam_r} Q h + P V,   P = (Q K^T) in_scale e^{gam_r - gam_i} where i <= r,
//     h' = e^{gam_last} h + K^T diag(in_scale e^{gam_last - gam}) V.
//
// One workgroup of eight waves owns 64 columns of S for a whole sequence (or segment) and keeps
// them in registers: wave w has columns 16 (w & 3) .. + 15 of rows KD/2 (w >> 2) .. .  The two
// waves of a column block add their halves of Q h through LDS, where the output is staged for
// rows of whole 128-byte lines.  The ten 16 x 16 tiles of P on and below the diagonal are spread
// over the waves and shared through LDS.  K, Q and V of the next chunk are copied global -> LDS
// meanwhile (bf16: two buffers).  Two barriers a chunk: P complete; output staged and the next
// chunk landed.
//
// rev: row r of a chunk is its r-th token from the end, and a row's gate is the next token's, so
// that the same code scans from the last token to the first.
//
// Precision: q, k and v in bf16 are exact operands.  h, P and the decayed V are fp32 and enter the
// bf16 matrix instructions in pieces of 8 bits each, x = hi + mid + lo to 2^-25 or hi + mid to
// 2^-17.  The state always takes three.  A bf16 output takes two of h and P: its own rounding is
// 2^-9.  An fp32 output, and the sums that gate gradients are differences of, take three.  fp32
// inputs use the fp32 matrix instruction.
#include "gdr_la.hpp"

namespace gdr {
namespace {

constexpr int NT = 512;   // threads
constexpr int BW = 64;    // columns of a workgroup

// A gate below this empties the state like this one: e^-104 is 0 in fp32.  (Sums of gates stay
// finite, and -inf may be given.)
constexpr float LOWEST_GATE = -104.f;

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
// small pieces first
template <int NP> __device__ __forceinline__ f32x4 mma(f32x4 c, const Pieces<bf16, NP> &a, const OpX &b) {
#pragma unroll
    for (int i = NP - 1; i >= 0; --i) c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.p[i], cat(b.b0, b.b1), c, 0, 0, 0);
    return c;
}
template <int NP> __device__ __forceinline__ f32x4 mma(f32x4 c, const OpX &a, const Pieces<bf16, NP> &b) {
#pragma unroll
    for (int i = NP - 1; i >= 0; --i) c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(cat(a.b0, a.b1), b.p[i], c, 0, 0, 0);
    return c;
}
template <int NP> __device__ __forceinline__ f32x4 mma(f32x4 c, const Pieces<float, NP> &a, const OpF &b) {
    return mma(c, a.x, b);
}
template <int NP> __device__ __forceinline__ f32x4 mma(f32x4 c, const OpF &a, const Pieces<float, NP> &b) {
    return mma(c, a, b.x);
}

// ------------------------------------------------------------ LDS layout
template <typename In, int KD, int NP, bool OUT> struct Lay {
    static constexpr bool BF = sizeof(In) == 2;
    static constexpr int ES = sizeof(In), NB = BF ? 2 : 1;
    static constexpr int KROW = KD * ES, VROW = BW * ES, PROW = CH * ES;
    static constexpr int KT = CH * KROW, VT = CH * VROW;
    static constexpr int OFF_K = 0, OFF_V = KT, OFF_Q = KT + VT, BUF = KT + VT + (OUT ? KT : 0);
    static constexpr int PPLANE = CH * PROW, NPL = BF ? NP : 1;
    static constexpr int OPLANE = CH * BW * 4;
    static constexpr int OFF_P = NB * BUF, OFF_O = OFF_P + (OUT ? NPL * PPLANE : 0), OFF_G = OFF_O + (OUT ? 2 * OPLANE : 0);
    static constexpr int GT = 7 * CH;  // floats of a chunk's gate table
    static constexpr int BYTES = OFF_G + 2 * GT * 4;
    static_assert(BYTES <= 160 * 1024, "LDS of a compute unit");
    using SK = Swz<KROW, KeyKQ>;
    using SV = Swz<VROW, KeyVP>;
    using SP = Swz<PROW, typename std::conditional<BF, KeyP, KeyVP>::type>;
    using SO = Swz<BW * 4>;
};
// gate table: running sums within a tile of 16 rows and their exponentials, decays from the
// chunk's start, to the chunk's end, and to the end of the tile 1, 2 or 3 tiles on
enum { G_LOC = 0, G_A = CH, G_START = 2 * CH, G_END = 3 * CH, G_TO = 4 * CH };

// one row's gate per lane -> the table; rows past n do not decay (their gate is 0) and add nothing
__device__ __forceinline__ void gate_table(float x, int n, float in_scale, float *t) {
    const int l = lane_id(), tile = l >> 4;
    x += dpp_mov<0x111>(x);  // row_shr 1, 2, 4, 8: running sums within 16 lanes
    x += dpp_mov<0x112>(x);
    x += dpp_mov<0x114>(x);
    x += dpp_mov<0x118>(x);
    auto total = [&](int i) { return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, x), i)); };
    const float t0 = total(15), t1 = total(31), t2 = total(47), t3 = total(63);
    const float before = tile == 0 ? 0.f : tile == 1 ? t0 : tile == 2 ? t0 + t1 : t0 + t1 + t2;
    const float mine = tile == 0 ? t0 : tile == 1 ? t1 : tile == 2 ? t2 : t3;
    const float next = tile == 0 ? t1 : tile == 1 ? t2 : t3, next2 = tile == 0 ? t2 : t3;
    const float rest = mine - x;  // to the end of the tile
    const float after = tile == 0 ? t1 + t2 + t3 : tile == 1 ? t2 + t3 : tile == 2 ? t3 : 0.f;
    t[G_LOC + l] = x;
    t[G_A + l] = fast_exp(x);
    t[G_START + l] = fast_exp(before + x);
    t[G_END + l] = l < n ? in_scale * fast_exp(rest + after) : 0.f;
    t[G_TO + l] = in_scale * fast_exp(rest);
    t[G_TO + CH + l] = in_scale * fast_exp(rest + next);
    t[G_TO + 2 * CH + l] = in_scale * fast_exp(rest + (next + next2));
}

__device__ __forceinline__ float sum8(float v) {  // over 8 lanes
    v += dpp_mov<0xB1>(v);
    v += dpp_mov<0x4E>(v);
    v += dpp_mov<0x141>(v);
    return v;
}

// OUT: with the output; else the end states of segments alone
template <typename In, int KD, int NP, bool OUT>
__global__ __launch_bounds__(NT) __attribute__((amdgpu_waves_per_eu(2, 2))) void gdr_la_scan_kernel(const LaParams p) {
    using Y = Lay<In, KD, NP, OUT>;
    using SK = typename Y::SK;
    using SV = typename Y::SV;
    using SP = typename Y::SP;
    using SO = typename Y::SO;
    using O = Ops<In>;
    using X = typename O::X;
    constexpr int ES = Y::ES, RT = KD / 32, U = KD / 64;  // 16-row tiles of a wave, pairs of them
    __shared__ __attribute__((aligned(16))) char lds[Y::BYTES];

    // ---------------------------------------------------------------- work item
    int id = xcd_remap(blockIdx.x, gridDim.x);
    const int cb = id % p.n_cb;
    id /= p.n_cb;
    const LaJob &J = p.job[id % p.n_jobs];
    id /= p.n_jobs;
    const int hv = id % p.s.Hv, item = id / p.s.Hv;
    int j = item, m = 0;
    if (p.split && !la_place(p.s, item, j, m)) return;
    int64_t bos, eos;
    la_bounds(p.s, j, bos, eos);
    const int len = (int)(eos - bos), nc = (len + CH - 1) / CH, rev = J.rev;
    const int first_place = p.s.seg_chunks ? la_first(bos, j, (int64_t)p.s.seg_chunks * CH) : 0;
    const int n_seg = p.split ? max(1, (nc + p.s.seg_chunks - 1) / p.s.seg_chunks) : 1;
    const int c_lo = p.split ? m * p.s.seg_chunks : 0, c_hi = p.split ? min(nc, c_lo + p.s.seg_chunks) : nc;
    const bool starts = m == (rev ? n_seg - 1 : 0), ends = m == (rev ? 0 : n_seg - 1);
    if (!OUT && ends) return;  // (no border after it)

    const int tid = threadIdx.x, l = lane_id(), n16 = ln16(), g = lg4();
    const int w = __builtin_amdgcn_readfirstlane(wave_id()), c4 = w & 3, half = w >> 2;
    const int64_t row0 = p.s.cu ? bos : 0, b0 = p.s.cu ? 0 : j;  // first token's row, batch row
    const char *kp = reinterpret_cast<const char *>(J.k) + (b0 * J.k_batch + row0 * J.k_row + (int64_t)(hv / J.k_div) * KD) * ES;
    const char *qp = reinterpret_cast<const char *>(J.q) + (b0 * J.q_batch + row0 * J.q_row + (int64_t)(hv / J.q_div) * KD) * ES;
    const char *vp = reinterpret_cast<const char *>(J.v) + (b0 * J.v_batch + row0 * J.v_row + (int64_t)(hv / J.v_div) * J.W + cb * BW) * ES;
    const float *gp = p.s.g + bos * p.s.g_tok + hv;

    // ------------------------------------------------------------------- states
    f32x4 h[RT];  // h[t][i]: row slot_base(half RT + t, g) + i, column 16 c4 + n16 of the block
    const int64_t KV = (int64_t)KD * J.W;
    const int col = cb * BW + 16 * c4 + n16;
    auto load_state = [&](const float *s) {
#pragma unroll
        for (int t = 0; t < RT; ++t) {
            const int r = slot_base(half * RT + t, g);
            if (J.trans) {
                h[t] = *reinterpret_cast<const f32x4 *>(s + (int64_t)col * KD + r);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) h[t][i] = s[(r + i) * J.W + col];
            }
        }
    };
    auto store_state = [&](float *s, float f) {
#pragma unroll
        for (int t = 0; t < RT; ++t) {
            const int r = slot_base(half * RT + t, g);
            if (J.trans) {
                *reinterpret_cast<f32x4 *>(s + (int64_t)col * KD + r) = f * h[t];
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) s[(r + i) * J.W + col] = f * h[t][i];
            }
        }
    };
    auto at_place = [&](float *s, int place) { return s + ((int64_t)place * p.s.Hv + hv) * KV; };
    const int64_t unit = (int64_t)j * p.s.Hv + hv;
    if (starts ? J.init != nullptr : OUT) {
        load_state(starts ? J.init + unit * KV : at_place(J.border, first_place + (rev ? m + 1 : m)));
    } else {
#pragma unroll
        for (int t = 0; t < RT; ++t) h[t] = zero4();
    }

    // ---------------------------------------------------------- a chunk's copies
    const int n_it = c_hi - c_lo;
    auto chunk_of = [&](int it) { return rev ? c_hi - 1 - it : c_lo + it; };
    auto copy_tile = [&](auto swz, const char *src, int64_t row, int nm1, char *dst, auto bytes) {
        using S = decltype(swz);
        constexpr int ROWB = S::CPR * 16, PIECES = decltype(bytes)::value / 1024;
        static_assert(PIECES % 8 == 0, "pieces spread over the waves");
#pragma unroll
        for (int i = 0; i < PIECES / 8; ++i) {
            const int piece = 8 * i + w, b = piece * 1024 + 16 * l, r = b / ROWB, pc = (b % ROWB) / 16;
            const int rr = min(r, nm1), tok = rev ? nm1 - rr : rr;  // rows past the end repeat the last one
            dma16(src + (uint32_t)(tok * (uint32_t)(row * ES) + 16 * S::chunk(r, pc)), dst + piece * 1024);
        }
    };
    auto issue = [&](int c, char *b) {
        const int64_t t0 = (int64_t)c * CH;
        const int nm1 = min(CH, len - (int)t0) - 1;
        copy_tile(SK{}, kp + t0 * J.k_row * ES, J.k_row, nm1, b + Y::OFF_K, std::integral_constant<int, Y::KT>{});
        copy_tile(SV{}, vp + t0 * J.v_row * ES, J.v_row, nm1, b + Y::OFF_V, std::integral_constant<int, Y::VT>{});
        if constexpr (OUT)
            copy_tile(SK{}, qp + t0 * J.q_row * ES, J.q_row, nm1, b + Y::OFF_Q, std::integral_constant<int, Y::KT>{});
    };
    // this lane's row's gate
    auto gate = [&](int c) {
        const int n = min(CH, len - c * CH), t = c * CH + (rev ? n - l : l);
        float x = 0.f;
        if (l < n && t < len) x = gp[(int64_t)t * p.s.g_tok];
        return x < LOWEST_GATE ? LOWEST_GATE : x;
    };
    float *gates = reinterpret_cast<float *>(lds + Y::OFF_G);
    constexpr int GW = 2;  // the wave that makes the gate tables (it has no score tile)
    float g_next = 0.f, whole = 1.f;

    // ------------------------------------------------------------------- output
    typedef typename Vec16<In>::type vec16;
    constexpr int EVN = 8 / Vec16<In>::n;
    vec16 ev[EVN];  // this thread's part of e for the chunk that is staged
    const int orow = tid >> 3, ocol = 8 * (tid & 7);
    auto row_token = [&](int c) {  // token of the staged row this thread stores, or -1
        const int n = min(CH, len - c * CH);
        return orow < n ? c * CH + (rev ? n - 1 - orow : orow) : -1;
    };
    auto fetch_e = [&](int c) {
        const int t = row_token(c);
        const In *e = reinterpret_cast<const In *>(J.e) + b0 * J.e_batch + row0 * J.e_row + (int64_t)(hv / J.e_div) * J.W +
                      cb * BW + ocol + (int64_t)max(t, 0) * J.e_row;
#pragma unroll
        for (int i = 0; i < EVN; ++i) ev[i] = *reinterpret_cast<const vec16 *>(e + i * Vec16<In>::n);
    };
    auto store_out = [&](int c) {
        const char *o0 = lds + Y::OFF_O, *o1 = o0 + Y::OPLANE;
        f32x4 y[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int off = SO::off(orow, 4 * (ocol + 4 * i));
            y[i] = J.out_scale * (*reinterpret_cast<const f32x4 *>(o0 + off) + *reinterpret_cast<const f32x4 *>(o1 + off));
        }
        const int t = row_token(c);
        if (J.dots) {
            float d = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) d = fmaf(y[i >> 2][i & 3], to_f32(ev[i / Vec16<In>::n][i % Vec16<In>::n]), d);
            d = sum8(d);
            if ((tid & 7) == 0 && t >= 0) J.dots[((int64_t)cb * p.s.Hv + hv) * p.tokens + bos + t] = d;
        }
        if (t < 0) return;
        const int64_t off = ((bos + t) * p.s.Hv + hv) * J.W + cb * BW + ocol;
        if (J.o_bf16) {
            __builtin_nontemporal_store(cat(narrow(y[0]), narrow(y[1])),
                                        reinterpret_cast<bf16x8 *>(reinterpret_cast<bf16 *>(J.o) + off));
        } else {
            float *o = reinterpret_cast<float *>(J.o) + off;
            __builtin_nontemporal_store(y[0], reinterpret_cast<f32x4 *>(o));
            __builtin_nontemporal_store(y[1], reinterpret_cast<f32x4 *>(o + 4));
        }
    };

    // ----------------------------------------------------------------- prologue
    char *pplane = lds + Y::OFF_P;
    if (n_it > 0) {
        issue(chunk_of(0), lds);
        if (w == GW) {
            gate_table(gate(chunk_of(0)), min(CH, len - chunk_of(0) * CH), J.in_scale, gates);
            if (n_it > 1) g_next = gate(chunk_of(1));
        }
        if constexpr (OUT) {
            // the tiles of P right of the diagonal that a 32-deep product reads: zero, never written
            constexpr int per = 16 * 16 * 2;  // elements of a plane
            for (int i = tid; i < per * Y::NPL; i += NT) {
                const int e = i % per, t = e >> 8, r = 32 * t + ((e >> 4) & 15), k = 32 * t + 16 + (e & 15);
                *reinterpret_cast<In *>(pplane + (i / per) * Y::PPLANE + SP::off(r, k * ES)) = In(0.f);
            }
        }
        wait_dma();
        lds_barrier();
    }

    // score tiles (row tile, key tile) of this wave: the waves whose half of P V is the shorter
    // one take two each
    constexpr int none = -1;
    const int tile0 = w == 4 ? 0x30 : w == 5 ? 0x32 : w == 6 ? 0x20 : w == 7 ? 0x22 : w == 0 ? 0x00 : w == 1 ? 0x11 : none;
    const int tile1 = w == 4 ? 0x31 : w == 5 ? 0x33 : w == 6 ? 0x21 : w == 7 ? 0x10 : none;

    for (int it = 0; it < n_it; ++it) {
        const int c = chunk_of(it);
        char *b = lds + (Y::NB == 2 ? (it & 1) * Y::BUF : 0);
        const char *Ks = b + Y::OFF_K, *Vs = b + Y::OFF_V, *Qs = b + Y::OFF_Q;
        const float *gt = gates + (it & 1) * Y::GT;
        if (Y::NB == 2 && it + 1 < n_it) issue(chunk_of(it + 1), lds + ((it + 1) & 1) * Y::BUF);
        if constexpr (OUT) {
            if (it > 0) store_out(chunk_of(it - 1));
            if (J.dots) fetch_e(c);
        }
        f32x4 o[4];
        X vo[2];
#pragma unroll
        for (int ip = 0; ip < 2; ++ip) vo[ip] = kt8<In, SV>(Vs, 32 * ip, 16 * c4, 4);
        if constexpr (OUT) {
            // P tiles
            auto score = [&](int tile) {
                const int rt = tile >> 4, kt = tile & 15;
                f32x4 s = zero4();
#pragma unroll
                for (int u = 0; u < KD / 32; ++u)
                    s = mma(s, frag8<In, SK>(Ks, 16 * kt + n16, (32 * u + 8 * g) * ES),
                            frag8<In, SK>(Qs, 16 * rt + n16, (32 * u + 8 * g) * ES));
                const int r = 16 * rt + n16, k0 = 16 * kt + 4 * g;  // s[i]: row r, key k0 + i
                if (rt == kt) {
                    const f32x4 gk = *reinterpret_cast<const f32x4 *>(gt + G_LOC + k0);
                    const float gr = gt[G_LOC + r];
#pragma unroll
                    for (int i = 0; i < 4; ++i) s[i] = 4 * g + i <= n16 ? s[i] * (J.in_scale * fast_exp(gr - gk[i])) : 0.f;
                } else {
                    s *= *reinterpret_cast<const f32x4 *>(gt + G_TO + (rt - kt - 1) * CH + k0) * gt[G_A + r];
                }
                const int off = SP::off(r, k0 * ES);
                if constexpr (Y::BF) {
                    bf16x4 x[NP];
                    pieces4<NP>(s, x);
#pragma unroll
                    for (int i = 0; i < NP; ++i) *reinterpret_cast<bf16x4 *>(pplane + i * Y::PPLANE + off) = x[i];
                } else {
                    *reinterpret_cast<f32x4 *>(pplane + off) = s;
                }
            };
            if (tile0 != none) score(tile0);
            if (tile1 != none) score(tile1);
            // this half's part of (Q h)^T: lane (token n16 of tile r, columns 4g ..)
#pragma unroll
            for (int r = 0; r < 4; ++r) o[r] = zero4();
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const Pieces<In, NP> hp = pieces8<In, NP>(h[2 * u], h[2 * u + 1]);
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    o[r] = mma(o[r], hp, frag8<In, SK>(Qs, 16 * r + n16, (half * (KD / 2) + 32 * u + 8 * g) * ES));
            }
#pragma unroll
            for (int r = 0; r < 4; ++r) o[r] *= gt[G_START + 16 * r + n16];
        }
        // the state at the chunk's end
        const float all = gt[G_START + CH - 1];
#pragma unroll
        for (int t = 0; t < RT; ++t) h[t] *= all;
        if (!OUT) whole *= all;
#pragma unroll
        for (int ip = 0; ip < 2; ++ip) {
            const f32x4 *e = reinterpret_cast<const f32x4 *>(gt + G_END + 32 * ip + 8 * g);
            f32x4 x0, x1;
            if constexpr (Y::BF) {
                x0 = widen(vo[ip].b0), x1 = widen(vo[ip].b1);
            } else {
                x0 = vo[ip].b0, x1 = vo[ip].b1;
            }
            const Pieces<In, 3> vd = pieces8<In, 3>(x0 * e[0], x1 * e[1]);
#pragma unroll
            for (int t = 0; t < RT; ++t) {
                const int tt = half * RT + t;
                h[t] = mma(h[t], kt8<In, SK>(Ks, 32 * ip, 32 * (tt >> 1) + 4 * (tt & 1), 8), vd);
            }
        }
        if (w == GW && it + 1 < n_it) {
            const int cn = chunk_of(it + 1);
            gate_table(g_next, min(CH, len - cn * CH), J.in_scale, gates + ((it + 1) & 1) * Y::GT);
            if (it + 2 < n_it) g_next = gate(chunk_of(it + 2));
        }
        if constexpr (OUT) {
            lds_barrier();  // P complete, the staged output stored
            // P V: a half of the keys each
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                if (r < 2 && half == 1) continue;
                const int off0 = SP::off(16 * r + n16, (32 * half + 8 * g) * ES);
                const X v = half ? vo[1] : vo[0];
                if constexpr (Y::BF) {
#pragma unroll
                    for (int i = NP - 1; i >= 0; --i)
                        o[r] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                            cat(v.b0, v.b1), *reinterpret_cast<const bf16x8 *>(pplane + i * Y::PPLANE + off0), o[r], 0, 0, 0);
                } else {
                    const int off1 = SP::off(16 * r + n16, (32 * half + 8 * g) * ES + 16);
                    o[r] = mma(o[r], v, OpF{*reinterpret_cast<const f32x4 *>(pplane + off0),
                                            *reinterpret_cast<const f32x4 *>(pplane + off1)});
                }
            }
            char *op = lds + Y::OFF_O + half * Y::OPLANE;
#pragma unroll
            for (int r = 0; r < 4; ++r) *reinterpret_cast<f32x4 *>(op + SO::off(16 * r + n16, 4 * (16 * c4 + 4 * g))) = o[r];
            // a border inside the scan
            if (J.border && !p.split) {
                const int after = rev ? c : c + 1;
                if (after % p.s.seg_chunks == 0 && after > 0 && after < nc)
                    store_state(at_place(J.border, first_place + after / p.s.seg_chunks), 1.f);
            }
        }
        wait_dma();
        lds_barrier();  // output staged, this buffer free, the next chunk landed
        if (Y::NB == 1 && it + 1 < n_it) {
            issue(chunk_of(it + 1), lds);
            wait_dma();
            lds_barrier();
        }
    }
    if constexpr (OUT) {
        if (n_it > 0) store_out(chunk_of(n_it - 1));
        if (ends && J.fin) {
            float f = 1.f;
            if (rev && len > 0) {
                const float x = gp[0];
                f = fast_exp(x < LOWEST_GATE ? LOWEST_GATE : x);
            }
            store_state(J.fin + unit * KV, f);
        }
        if (ends && J.border_fin) store_state(at_place(J.border_fin, first_place), 1.f);
    } else {
        store_state(at_place(J.border, first_place + (rev ? m : m + 1)), 1.f);
        if (cb == 0 && tid == 0) J.decays[(int64_t)(first_place + m) * p.s.Hv + hv] = whole;
    }
}

template <typename In, int KD, int NP, bool OUT>
hipError_t launch(const LaParams &p, int items, hipStream_t s) {
    launch_k(gdr_la_scan_kernel<In, KD, NP, OUT>, dim3((uint32_t)items * p.s.Hv * p.n_jobs * p.n_cb), dim3(NT), 0, s, p);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_la_scan(Dt dt, int KD, bool fine, const LaParams &p, int items, hipStream_t s) {
    if (dt == Dt::F32) return KD == 128 ? launch<float, 128, 1, true>(p, items, s) : launch<float, 64, 1, true>(p, items, s);
    if (fine) return KD == 128 ? launch<bf16, 128, 3, true>(p, items, s) : launch<bf16, 64, 3, true>(p, items, s);
    return KD == 128 ? launch<bf16, 128, 2, true>(p, items, s) : launch<bf16, 64, 2, true>(p, items, s);
}

hipError_t launch_la_states(Dt dt, int KD, const LaParams &p, int items, hipStream_t s) {
    if (dt == Dt::F32) return KD == 128 ? launch<float, 128, 1, false>(p, items, s) : launch<float, 64, 1, false>(p, items, s);
    return KD == 128 ? launch<bf16, 128, 1, false>(p, items, s) : launch<bf16, 64, 1, false>(p, items, s);
}

}  // namespace gdr
