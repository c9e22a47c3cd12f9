// gdr_step: the recurrent form of the gated delta rule, a token at a time on a
// pool of states; gdr_tree_accept: the same over the tokens of an accepted path;
// gdr_la_step: the recurrent form of linear attention, the rule without its correction.
//
// Per (sequence, v head), with the state h (K x V, fp32):
//     u = beta (v - e^g k h),   h <- e^g h + k u^T,   o = scale q h.
// Columns of h are independent, and both products are taken of the old state:
// q h_new = e^g q h + (q . k) u, so that one pass over the state's registers and
// one sum over the lanes serve u and o together.  Without the correction u is v.
//
// A wave holds K rows x 32 columns of the state in registers over all of the
// sequence's tokens: lane l has columns 4 (l & 7) .. + 3 of rows R (l >> 3) ..
// + R - 1, R = K / 8, so that a load or store of the state is 8 rows x 128 bytes
// and the rows of k and q that a lane needs are consecutive.  No LDS, no barriers (but for
// a long list of slots).
//
// Bound by the state's traffic, 8 K V bytes per head and call.  256 sequences of 32 heads
// (K = V = 128, 1.07 GB) take 185 us, 5.8 TB/s; an in-place multiplication of 1 GB runs at
// 6.0.  The loads and stores of the state are nontemporal and an XCD takes runs of 8 heads:
// 205 us with cached accesses, 189 with heads dealt singly.  Waves of 16 columns (twice as
// many) take 269 us there and gain 0.2 us at one sequence (both of one token).  A token beyond
// the first adds about 1 us to a sequence: some 270 fp32 instructions of a wave.
#include "gdr_pool.hpp"

namespace gdr {
namespace {

// Sums over the lanes with the same l & 7 (the row groups).  v_permlane32_swap_b32 exchanges
// the upper half of its first register with the lower half of its second, v_permlane16_swap_b32
// the odd rows of 16 lanes of the first with the even ones of the second: two values are
// reduced in one exchange and one addition, and lie in a half (a row) of the lanes each.
struct Swapped {
    float a, b;
};
__device__ __forceinline__ Swapped swap32(float a, float b) {
    const auto r = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b), false, false);
    const uint32_t r0 = r[0], r1 = r[1];
    return {__builtin_bit_cast(float, r0), __builtin_bit_cast(float, r1)};
}
__device__ __forceinline__ Swapped swap16(float a, float b) {
    const auto r = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b), false, false);
    const uint32_t r0 = r[0], r1 = r[1];
    return {__builtin_bit_cast(float, r0), __builtin_bit_cast(float, r1)};
}
// a second register with x's value, which the exchange writes too
__device__ __forceinline__ float twin(float x) {
    asm volatile("" : "+v"(x));
    return x;
}
// column of the lane's four whose sum it gets
__device__ __forceinline__ int my_column(int l) { return (l >> 5 & 1) | (l >> 3 & 2); }
__device__ __forceinline__ float sum_columns(f32x4 x) {
    const Swapped p = swap32(x[0], x[1]), q = swap32(x[2], x[3]);
    const Swapped y = swap16(p.a + p.b, q.a + q.b);
    const float z = y.a + y.b;
    return z + dpp_mov<0x128>(z);  // row_ror:8
}
__device__ __forceinline__ float sum_all(float x) {
    x += dpp_mov<0x128>(x);
    const Swapped y = swap16(x, twin(x));
    x = y.a + y.b;
    const Swapped z = swap32(x, twin(x));
    return z.a + z.b;
}
// every column's value from the lanes that have it
__device__ __forceinline__ f32x4 gather_columns(float x) {
    const Swapped y = swap16(x, twin(x));
    const Swapped lo = swap32(y.a, twin(y.a)), hi = swap32(y.b, twin(y.b));
    return f32x4{lo.a, lo.b, hi.a, hi.b};
}

// R consecutive inputs
template <typename In, int R> struct Rows {
    typename Vec16<In>::type x[R / Vec16<In>::n];
    __device__ __forceinline__ void load(const In *p) {
#pragma unroll
        for (int i = 0; i < R / Vec16<In>::n; ++i)
            x[i] = *reinterpret_cast<const typename Vec16<In>::type *>(p + i * Vec16<In>::n);
    }
    __device__ __forceinline__ float operator[](int r) const {
        return to_f32(x[r / Vec16<In>::n][r % Vec16<In>::n]);
    }
};

template <typename In, int R> struct Token {
    Rows<In, R> k, q;
    In v;
    float g, beta;
};

enum class Rule { DELTA, ACCEPT, DECAY };

template <typename In, typename Out, int K, Rule RULE>
__global__ __launch_bounds__(256) void gdr_step_kernel(PoolParams p, int V) {
    constexpr int R = K / 8;
    constexpr bool ACCEPT = RULE == Rule::ACCEPT, DECAY = RULE == Rule::DECAY;
    const int unit = xcd_runs(blockIdx.x, gridDim.x), vt = __builtin_amdgcn_readfirstlane(wave_id());
    const int j = unit / p.Hv, hv = unit - j * p.Hv, hq = hv / (p.Hv / p.Hq);
    const int l = lane_id(), col = vt * 32 + 4 * (l & 7), row0 = R * (l >> 3), mine = col + my_column(l);
    int64_t bos, eos;
    token_range(p, j, bos, eos);
    if (bos >= eos) return;
    const int slot = slot_of(p, j);
    Out *o = reinterpret_cast<Out *>(p.o) + hv * V + mine;
    const bool writes = (l & 8) == 0;
    uint64_t path = 0;  // the accepted nodes
    if constexpr (ACCEPT) {
        if (slot < 0 || eos - bos > TREE_MAX) return;
        const int n = (int)(eos - bos);
        const int parent = l < n ? p.parents[bos + l] : -1;
        int node = p.accepted[j];
        if (node >= n) node = -1;
        while (node >= 0) {  // a parent that is no earlier node counts as -1: at most n steps
            path |= 1ull << node;
            const int up = __builtin_amdgcn_readlane(parent, node);
            node = up < node ? up : -1;
        }
        if (!path) return;
    }
    auto skip = [&] {
        if (!ACCEPT && writes)
            for (int64_t i = bos; i < eos; ++i) o[i * p.Hv * V] = (Out)0.f;
    };
    if (slot < 0) return skip();

    float *h0 = p.states + (int64_t)slot * p.slot_stride + ((int64_t)hv * K + row0) * V + col;
    f32x4 h[R];
#pragma unroll
    for (int r = 0; r < R; ++r) h[r] = load4_once(h0 + r * V);

    const In *kp = reinterpret_cast<const In *>(p.k) + hq * K + row0;
    const In *qp = reinterpret_cast<const In *>(p.q) + hq * K + row0;
    const In *vp = reinterpret_cast<const In *>(p.v) + hv * V + mine;
    Token<In, R> now, next;
    auto fetch = [&](Token<In, R> &t, int64_t i) {
        t.k.load(kp + row_offset(p, j, i, p.k_batch, p.k_row));
        if constexpr (!ACCEPT) t.q.load(qp + row_offset(p, j, i, p.q_batch, p.q_row));
        t.v = vp[row_offset(p, j, i, p.v_batch, p.v_row)];
        t.g = p.g[(DECAY ? i * p.g_tok : i * p.Hv) + hv];
        if constexpr (!DECAY) t.beta = p.beta[i * p.Hv + hv];
    };
    // every rounding is written out (no contraction by the compiler), so that an acceptance
    // and the recurrent form on the same tokens agree to the bit
    auto step = [&](const Token<In, R> &t, int64_t i) {
#pragma clang fp contract(off)
        f32x4 kh = zero4(), qh = zero4();
        float qk = 0.f;
#pragma unroll
        for (int r = 0; r < R; ++r) {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                if constexpr (!DECAY) kh[c] = __builtin_fmaf(t.k[r], h[r][c], kh[c]);
                if constexpr (!ACCEPT) qh[c] = __builtin_fmaf(t.q[r], h[r][c], qh[c]);
            }
            if constexpr (!ACCEPT) qk = __builtin_fmaf(t.q[r], t.k[r], qk);
        }
        // full-precision exponential: its error would otherwise grow with every token
        const float eg = expf(t.g);
        const float u = DECAY ? to_f32(t.v) : t.beta * __builtin_fmaf(-eg, sum_columns(kh), to_f32(t.v));
        const f32x4 us = gather_columns(u);
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int c = 0; c < 4; ++c) h[r][c] = __builtin_fmaf(t.k[r], us[c], eg * h[r][c]);
        if constexpr (!ACCEPT) {
            const float y = p.scale * __builtin_fmaf(sum_all(qk), u, eg * sum_columns(qh));
            if (writes) o[i * p.Hv * V] = (Out)y;
        }
    };
    fetch(now, ACCEPT ? bos + __builtin_ctzll(path) : bos);
    // with the loads in flight: a skipped sequence's are not used
    if (slot_taken(p, j, slot)) return skip();
    // the next token's loads are in flight during this one's work.  The last token fetches itself
    // again: a condition would end the block of instructions, and the loads be waited for there
    if constexpr (ACCEPT) {
        for (bool more = true; more;) {
            const int64_t i = bos + __builtin_ctzll(path);
            more = (path & (path - 1)) != 0;
            if (more) path &= path - 1;
            fetch(next, bos + __builtin_ctzll(path));
            step(now, i);
            now = next;
        }
    } else {
        for (int64_t i = bos; i < eos; ++i) {
            fetch(next, min(i + 1, eos - 1));
            step(now, i);
            now = next;
        }
    }
#pragma unroll
    for (int r = 0; r < R; ++r) store4_once(h0 + r * V, h[r]);
}

template <typename In, typename Out, Rule RULE>
hipError_t launch(int K, int V, const PoolParams &p, hipStream_t s) {
    // a head's waves in one workgroup share its k and q rows in the L1
    const int block = 64 * (V / 32);
    const dim3 grid((uint32_t)p.n_seq * p.Hv);
    // LDS that no kernel uses holds a compute unit to eight waves of 128 rows, the 128 KB in
    // flight at which HBM is fastest: 256 sequences of 32 heads take 185 us, 192 with the twelve
    // that the registers leave room for.  With 64 rows sixteen waves are (11.5 us for 4096
    // waves, 14.5 for eight at a time), and an acceptance does not mind.
    const uint32_t lds = RULE == Rule::ACCEPT || K == 64 ? 0 : V == 128 ? 54 << 10 : 33 << 10;
    if (K == 128)
        launch_k(gdr_step_kernel<In, Out, 128, RULE>, grid, dim3(block), lds, s, p, V);
    else
        launch_k(gdr_step_kernel<In, Out, 64, RULE>, grid, dim3(block), lds, s, p, V);
    return hipGetLastError();
}

}  // namespace

template <Rule RULE> static hipError_t launch_rule(Dt dt, Dt out, int K, int V, const PoolParams &p, hipStream_t s) {
    if (dt == Dt::BF16)
        return out == Dt::BF16 ? launch<bf16, bf16, RULE>(K, V, p, s) : launch<bf16, float, RULE>(K, V, p, s);
    return out == Dt::BF16 ? launch<float, bf16, RULE>(K, V, p, s) : launch<float, float, RULE>(K, V, p, s);
}

hipError_t launch_step(Dt dt, Dt out, int K, int V, const PoolParams &p, hipStream_t s) {
    return launch_rule<Rule::DELTA>(dt, out, K, V, p, s);
}

hipError_t launch_la_step(Dt dt, Dt out, int K, int V, const PoolParams &p, hipStream_t s) {
    return launch_rule<Rule::DECAY>(dt, out, K, V, p, s);
}

hipError_t launch_accept(Dt dt, int K, int V, const PoolParams &p, hipStream_t s) {
    return dt == Dt::BF16 ? launch<bf16, float, Rule::ACCEPT>(K, V, p, s) : launch<float, float, Rule::ACCEPT>(K, V, p, s);
}

}  // namespace gdr
