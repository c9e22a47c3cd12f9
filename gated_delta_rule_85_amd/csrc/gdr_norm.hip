// gdr_group_norm: every token's groups of channels normalised, with weight and bias, and an
// activation: of a gate that multiplies the result, or of the result itself.
//
//     n = (x - mean) rstd,  y = n w + b,  out = y act(gate)  or  act(y);
// without centering, n = x / sqrt(mean(x^2) + eps).
//
// A group's values stay in registers: the mean first, then the mean square of what is left, so that
// nothing cancels.  Bound by memory: x and gate read once, out written once.
#include "gdr_norm.hpp"

namespace gdr {
namespace {

template <typename X, typename Z, typename Y, int VEC, int NE>
__global__ __launch_bounds__(NORM_THREADS) void gdr_norm_kernel(NormParams p, bool wide) {
    __shared__ float lds[2][4];
    const NormPlace at(p);
    if (!at.active) return;  // (never of a wide group)
    const int64_t C = (int64_t)p.groups * p.D, c0 = (int64_t)at.group * p.D;
    bool valid[NE / VEC];
    float w[NE], b[NE];
#pragma unroll
    for (int v = 0; v < NE / VEC; ++v) {
        const int c = norm_channel<VEC>(v * VEC, p.lanes, at.r);
        valid[v] = c < p.D;
#pragma unroll
        for (int i = 0; i < VEC; ++i) w[v * VEC + i] = 1.f, b[v * VEC + i] = 0.f;
        if (valid[v] && p.weight) norm_load<float, VEC>(p.weight + c0 + c, w + v * VEC);
        if (valid[v] && p.bias) norm_load<float, VEC>(p.bias + c0 + c, b + v * VEC);
    }
    int turn = 0;  // two places in turn: between two writes of one lies a barrier after its reads
    auto sum = [&](float v) {
        turn ^= 1;
        return wide ? norm_sum<true>(v, p.lanes, lds[turn]) : norm_sum<false>(v, p.lanes, lds[turn]);
    };
    const float per_channel = 1.f / p.D;
    for (int64_t t = (int64_t)blockIdx.y * at.per + at.sub; t < p.M; t += (int64_t)gridDim.y * at.per) {
        const X *x = static_cast<const X *>(p.x) + t * p.x_row + c0;
        const Z *z = static_cast<const Z *>(p.gate) + t * p.gate_row + c0;
        Y *o = static_cast<Y *>(p.out) + t * C + c0;
        float n[NE], a[NE];
#pragma unroll
        for (int v = 0; v < NE / VEC; ++v) {
#pragma unroll
            for (int i = 0; i < VEC; ++i) n[v * VEC + i] = a[v * VEC + i] = 0.f;
            if (!valid[v]) continue;
            const int c = norm_channel<VEC>(v * VEC, p.lanes, at.r);
            norm_load<X, VEC>(x + c, n + v * VEC);
            if (p.gate) norm_load<Z, VEC>(z + c, a + v * VEC);
        }
        float total = 0.f;
        if (p.center) {
#pragma unroll
            for (int i = 0; i < NE; ++i) total += n[i];
            const float mean = sum(total) * per_channel;
#pragma unroll
            for (int i = 0; i < NE; ++i) n[i] = valid[i / VEC] ? n[i] - mean : 0.f;
        }
        total = 0.f;
#pragma unroll
        for (int i = 0; i < NE; ++i) total = fmaf(n[i], n[i], total);
        const float rstd = rsqrtf(fmaf(sum(total), per_channel, p.eps));
#pragma unroll
        for (int v = 0; v < NE / VEC; ++v) {
            if (!valid[v]) continue;
            float y[VEC];
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                const int k = v * VEC + i;
                y[i] = fmaf(n[k] * rstd, w[k], b[k]);
                y[i] = p.gate ? y[i] * norm_act(p.act, a[k]) : norm_act(p.act, y[i]);
            }
            norm_store<Y, VEC>(o + norm_channel<VEC>(v * VEC, p.lanes, at.r), y);
        }
    }
}

template <typename X, typename Z, typename Y, int VEC, int NE> struct Launch {
    static hipError_t go(NormGrid g, const NormParams &p, hipStream_t s) {
        launch_k(gdr_norm_kernel<X, Z, Y, VEC, NE>, dim3(g.x, g.y), dim3(NORM_THREADS), 0, s, p, p.lanes > 64);
        return hipGetLastError();
    }
};

}  // namespace

hipError_t launch_norm(Dt x, Dt gate, Dt out, NormVariant v, NormGrid g, const NormParams &p, hipStream_t s) {
    return norm_types<Launch>(x, gate, out, v, g, p, s);
}

}  // namespace gdr
