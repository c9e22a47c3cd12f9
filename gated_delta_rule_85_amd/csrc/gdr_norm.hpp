// Group norm with an activation (gdr_group_norm, gdr_group_norm_bwd): parameter block, thread map
// and element functions that both directions share.
#pragma once

#include "gdr_kernels.hpp"

namespace gdr {

constexpr int NORM_WIDTH_MAX = 8192;  // channels of a group
constexpr int NORM_THREADS = 256;

// A group's channels are spread over `lanes` lanes (a power of two up to 64, or the workgroup's
// 256), and a token takes groups x lanes places.  A workgroup has 256 places: of several tokens,
// of one, or a part of one's.  A thread keeps its channels over all of its tokens.
struct NormParams {
    const void *x, *gate, *dout;
    const float *weight, *bias;
    void *out, *dx, *dgate;
    float *part_w, *part_b;  // [gridDim.y][C] sums over a workgroup's tokens, or null
    int64_t M, x_row, gate_row;  // tokens; elements between tokens
    int groups, D, lanes, act, center;
    float eps;
};

enum { ACT_NONE = 0, ACT_SILU = 1, ACT_SIGMOID = 2 };

// how a launch spreads the tokens: x blocks of places, y workgroups along the tokens, `per` tokens
// of a workgroup at a time
struct NormGrid {
    uint32_t x, y;
    int per;
};
inline NormGrid norm_grid(int64_t M, int64_t groups, int lanes, int64_t workgroups) {
    const int64_t places = groups * lanes, x = (places + NORM_THREADS - 1) / NORM_THREADS;
    const int64_t per = places <= NORM_THREADS ? NORM_THREADS / places : 1;
    int64_t y = (M + per - 1) / per, most = (workgroups + x - 1) / x;
    if (y > most) y = most;
    return {(uint32_t)x, (uint32_t)(y < 1 ? 1 : y), (int)per};
}

// N values of a row as they lie in memory, read or written once: past the caches
template <typename T, int N> struct NormRaw;
template <typename T> struct NormRaw<T, 1> {
    T x;
    __device__ __forceinline__ void load(const T *p) { x = *p; }
    __device__ __forceinline__ float get(int) const { return to_f32(x); }
};
template <typename T> struct NormRaw<T, 8> {
    typedef typename Vec16<T>::type vec;
    static constexpr int n = Vec16<T>::n;
    vec x[8 / n];
    __device__ __forceinline__ void load(const T *p) {
#pragma unroll
        for (int v = 0; v < 8 / n; ++v) x[v] = __builtin_nontemporal_load(reinterpret_cast<const vec *>(p + v * n));
    }
    __device__ __forceinline__ float get(int i) const { return to_f32(x[i / n][i % n]); }
};
template <typename T> __device__ __forceinline__ void norm_store8(T *p, const float *y) {
    if constexpr (sizeof(T) == 2) {
        typedef float f32x8 __attribute__((ext_vector_type(8)));
        const f32x8 x = {y[0], y[1], y[2], y[3], y[4], y[5], y[6], y[7]};
        __builtin_nontemporal_store(__builtin_convertvector(x, bf16x8), reinterpret_cast<bf16x8 *>(p));
    } else {
        __builtin_nontemporal_store(f32x4{y[0], y[1], y[2], y[3]}, reinterpret_cast<f32x4 *>(p));
        __builtin_nontemporal_store(f32x4{y[4], y[5], y[6], y[7]}, reinterpret_cast<f32x4 *>(p + 4));
    }
}

// the activation of z, and its slope
__device__ __forceinline__ float norm_sigmoid(float z) { return __builtin_amdgcn_rcpf(1.f + fast_exp(-z)); }
__device__ __forceinline__ float norm_act(int act, float z) {
    if (act == ACT_NONE) return z;
    const float s = norm_sigmoid(z);
    return act == ACT_SILU ? z * s : s;
}
__device__ __forceinline__ float norm_act(int act, float z, float &slope) {
    if (act == ACT_NONE) {
        slope = 1.f;
        return z;
    }
    const float e = fast_exp(-z), s = __builtin_amdgcn_rcpf(1.f + e);
    // (the sigmoid's own slope by 1 - s = e s where s is near 1)
    slope = act == ACT_SILU ? fmaf(s * z, 1.f - s, s) : s * (z > 0.f ? e * s : 1.f - s);
    return act == ACT_SILU ? z * s : s;
}

// sum over a group's lanes; WIDE: of the workgroup's four waves
template <bool WIDE> __device__ __forceinline__ float norm_sum(float v, int lanes, float *lds) {
    if constexpr (WIDE) {
#pragma unroll
        for (int s = 32; s; s >>= 1) v += __shfl_xor(v, s);
        if (lane_id() == 0) lds[wave_id()] = v;
        __syncthreads();
        return (lds[0] + lds[1]) + (lds[2] + lds[3]);
    } else {
        for (int s = 1; s < lanes; s <<= 1) v += __shfl_xor(v, s);
        return v;
    }
}

// a thread's place
struct NormPlace {
    int sub, group, r, per;  // token of the workgroup's, group, lane of the group, tokens at a time
    bool active;
    __device__ __forceinline__ NormPlace(const NormParams &p) {
        const int places = p.groups * p.lanes, tid = threadIdx.x;
        int at = (int)blockIdx.x * NORM_THREADS + tid;
        sub = 0, per = 1;
        if (places <= NORM_THREADS) {
            per = NORM_THREADS / places;
            sub = tid / places;
            at = tid - sub * places;
        }
        active = sub < per && at < places;
        group = active ? at / p.lanes : 0;
        r = at & (p.lanes - 1);
    }
};

// A thread's channels: pieces of VEC, the lanes' pieces next to each other.  Pieces of 8 lie at multiples
// of 8 in the row; where a group does not (RAGGED), its first and last one hold another group's
// channels too, whose values (whatever they are) are taken as zero and never written: 5001 tokens of 8
// groups of 325 channels (bf16) forward in 29 us, with single channels 42 us.
template <int VEC, int NE, bool RAGGED> struct NormChannels {
    static constexpr int NV = NE / VEC;
    int at[NV];          // first channel of piece v in the row; past the group's end where there is none
    int from[NV], to[NV];  // its channels that are the group's (RAGGED)
    bool valid[NV];
    __device__ __forceinline__ NormChannels(const NormParams &p, const NormPlace &pl) {
        const int first = pl.group * p.D, shift = RAGGED ? first & 7 : 0;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c = (v * p.lanes + pl.r) * VEC - shift;  // in the group
            at[v] = first + c;
            valid[v] = pl.active && c < p.D;
            from[v] = max(0, -c), to[v] = min(VEC, p.D - c);
        }
    }
    // whether value i (of piece i / VEC) is the group's
    __device__ __forceinline__ bool has(int i) const {
        const int v = i / VEC, k = i % VEC;
        return RAGGED ? valid[v] && k >= from[v] && k < to[v] : valid[v];
    }
    template <typename T> __device__ __forceinline__ void store(T *row, int v, const float *y) const {
        if (VEC == 1) {
            row[at[v]] = (T)y[0];
        } else if (!RAGGED || (from[v] == 0 && to[v] == VEC)) {
            norm_store8(row + at[v], y);
        } else {
#pragma unroll
            for (int k = 0; k < VEC; ++k)
                if (k >= from[v] && k < to[v]) row[at[v] + k] = (T)y[k];
        }
    }
    template <typename T> __device__ __forceinline__ void load(const T *row, NormRaw<T, VEC> (&x)[NV]) const {
#pragma unroll
        for (int v = 0; v < NV; ++v)
            if (valid[v]) x[v].load(row + at[v]);
    }
    template <typename T> __device__ __forceinline__ void values(const NormRaw<T, VEC> (&x)[NV], float *y) const {
#pragma unroll
        for (int i = 0; i < NE; ++i) y[i] = has(i) ? x[i / VEC].get(i % VEC) : 0.f;
    }
    // of weight or bias, or `none`
    __device__ __forceinline__ void parameters(const float *row, float none, float *y) const {
#pragma unroll
        for (int i = 0; i < NE; ++i) y[i] = !has(i) ? 0.f : row ? row[at[i / VEC] + i % VEC] : none;
    }
};

struct NormVariant {
    int vec, values, lanes;
    bool ragged;
};
// Pieces of 8 where the rows allow them and a workgroup has a place for all that a group may touch (1025
// of them for 8187, 8189, 8190 and 8191 channels), else single channels.  A ragged group begins up to
// 8 - (D & -D) channels past a multiple of 8
inline NormVariant norm_variant(int64_t D, bool aligned) {
    const bool ragged = aligned && D % 8 != 0;
    const int64_t width = ragged ? (D + 8 - (D & -D) + 7) / 8 * 8 : D;  // of the pieces that it may touch
    if (aligned && width <= NORM_WIDTH_MAX) {
        if (width > 512) return {8, width <= 2048 ? 8 : width <= 4096 ? 16 : 32, NORM_THREADS, ragged};
        int lanes = 1;
        while (lanes * 8 < width) lanes <<= 1;
        return {8, 8, lanes, ragged};
    }
    if (D > 512) return {1, D <= 2048 ? 8 : 32, NORM_THREADS, false};
    int lanes = 8;
    while (lanes * 8 < D) lanes <<= 1;
    return {1, 8, lanes, false};
}

hipError_t launch_norm(Dt x, Dt gate, Dt out, NormVariant v, NormGrid g, const NormParams &p, hipStream_t s);
hipError_t launch_norm_bwd(Dt x, Dt gate, Dt out, NormVariant v, NormGrid g, const NormParams &p, hipStream_t s);
// w[c], b[c] (either may be null) = sums over the parts of part_w[.][c], part_b[.][c]
hipError_t launch_norm_sum(const float *part_w, const float *part_b, float *w, float *b, int64_t parts, int64_t C, hipStream_t s);

// types and variant -> instantiation
template <template <typename, typename, typename, int, int, bool> class Launch, typename X, typename Z, typename Y>
hipError_t norm_values(NormVariant v, NormGrid g, const NormParams &p, hipStream_t s) {
    if (v.vec == 1) return v.values == 8 ? Launch<X, Z, Y, 1, 8, false>::go(g, p, s) : Launch<X, Z, Y, 1, 32, false>::go(g, p, s);
    if (v.values == 8) return v.ragged ? Launch<X, Z, Y, 8, 8, true>::go(g, p, s) : Launch<X, Z, Y, 8, 8, false>::go(g, p, s);
    // (few groups are wider than 2048: one kernel for both)
    return v.values == 16 ? Launch<X, Z, Y, 8, 16, true>::go(g, p, s) : Launch<X, Z, Y, 8, 32, true>::go(g, p, s);
}
template <template <typename, typename, typename, int, int, bool> class Launch>
hipError_t norm_types(Dt x, Dt z, Dt y, NormVariant v, NormGrid g, const NormParams &p, hipStream_t s) {
    const int t = (x == Dt::F32) << 2 | (z == Dt::F32) << 1 | (y == Dt::F32);
    switch (t) {
        case 0: return norm_values<Launch, bf16, bf16, bf16>(v, g, p, s);
        case 1: return norm_values<Launch, bf16, bf16, float>(v, g, p, s);
        case 2: return norm_values<Launch, bf16, float, bf16>(v, g, p, s);
        case 3: return norm_values<Launch, bf16, float, float>(v, g, p, s);
        case 4: return norm_values<Launch, float, bf16, bf16>(v, g, p, s);
        case 5: return norm_values<Launch, float, bf16, float>(v, g, p, s);
        case 6: return norm_values<Launch, float, float, bf16>(v, g, p, s);
        default: return norm_values<Launch, float, float, float>(v, g, p, s);
    }
}

}  // namespace gdr
