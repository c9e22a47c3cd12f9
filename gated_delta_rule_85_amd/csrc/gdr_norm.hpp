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
    float *part_w, *part_b;  // [parts][C] sums of a workgroup's tokens, or null
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

template <typename T, int N> __device__ __forceinline__ void norm_load(const T *p, float *y) {
    if constexpr (N == 1) {
        y[0] = to_f32(*p);
    } else {
        constexpr int n = Vec16<T>::n;
#pragma unroll
        for (int v = 0; v < N / n; ++v) {
            const typename Vec16<T>::type x = *reinterpret_cast<const typename Vec16<T>::type *>(p + v * n);
#pragma unroll
            for (int i = 0; i < n; ++i) y[v * n + i] = to_f32(x[i]);
        }
    }
}
template <typename T, int N> __device__ __forceinline__ void norm_store(T *p, const float *y) {
    if constexpr (N == 1) {
        *p = (T)y[0];
    } else if constexpr (sizeof(T) == 2) {
        typedef float f32x8 __attribute__((ext_vector_type(8)));
        const f32x8 x = {y[0], y[1], y[2], y[3], y[4], y[5], y[6], y[7]};
        *reinterpret_cast<bf16x8 *>(p) = __builtin_convertvector(x, bf16x8);
    } else {
        *reinterpret_cast<f32x4 *>(p) = f32x4{y[0], y[1], y[2], y[3]};
        *reinterpret_cast<f32x4 *>(p + 4) = f32x4{y[4], y[5], y[6], y[7]};
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
    const float s = norm_sigmoid(z);
    slope = act == ACT_SILU ? fmaf(s * z, 1.f - s, s) : s * (1.f - s);
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

// Channel of a thread's value i within its group: VEC 8: pieces of 8, the lanes' pieces next to
// each other; VEC 1: one by one
template <int VEC> __device__ __forceinline__ int norm_channel(int i, int lanes, int r) {
    return VEC == 8 ? ((i >> 3) * lanes + r) * 8 + (i & 7) : i * lanes + r;
}

struct NormVariant {
    int vec, values, lanes;
};
// Pieces of 8 where the width and every row allow them, else single channels
inline NormVariant norm_variant(int64_t D, bool aligned) {
    if (aligned && D % 8 == 0) {
        if (D > 512) return {8, D <= 2048 ? 8 : D <= 4096 ? 16 : 32, NORM_THREADS};
        int lanes = 1;
        while (lanes * 8 < D) lanes <<= 1;
        return {8, 8, lanes};
    }
    if (D > 512) return {1, D <= 2048 ? 8 : 32, NORM_THREADS};
    int lanes = 8;
    while (lanes * 8 < D) lanes <<= 1;
    return {1, 8, lanes};
}

hipError_t launch_norm(Dt x, Dt gate, Dt out, NormVariant v, NormGrid g, const NormParams &p, hipStream_t s);
hipError_t launch_norm_bwd(Dt x, Dt gate, Dt out, NormVariant v, NormGrid g, const NormParams &p, hipStream_t s);
// out[c] = sum over the parts of part[.][c]
hipError_t launch_norm_sum(const float *part, float *out, int64_t parts, int64_t C, hipStream_t s);

// types and variant -> instantiation
template <template <typename, typename, typename, int, int> class Launch, typename X, typename Z, typename Y>
hipError_t norm_values(NormVariant v, NormGrid g, const NormParams &p, hipStream_t s) {
    if (v.vec == 1) return v.values == 8 ? Launch<X, Z, Y, 1, 8>::go(g, p, s) : Launch<X, Z, Y, 1, 32>::go(g, p, s);
    if (v.values == 8) return Launch<X, Z, Y, 8, 8>::go(g, p, s);
    return v.values == 16 ? Launch<X, Z, Y, 8, 16>::go(g, p, s) : Launch<X, Z, Y, 8, 32>::go(g, p, s);
}
template <template <typename, typename, typename, int, int> class Launch>
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
