// gdr_group_norm_bwd: gradients of the group norm with its activation.
//
// With n and y as in the forward, which is computed again from x (its statistics cost no pass of
// their own: the group is in registers):
//     with a gate:  dgate = dout y act'(gate),  dy = dout act(gate);   else  dy = dout act'(y);
//     dw = sum over tokens dy n,  db = sum over tokens dy,  dn = dy w,
//     dx = rstd (dn - n mean(dn n) - mean(dn)),  the last term where the norm is centred.
// A thread keeps its channels over its tokens and their dw and db in registers; the sums of the
// workgroups are added in a second kernel, in the order of the workgroups.
#include "gdr_norm.hpp"

namespace gdr {
namespace {

template <typename X, typename Z, typename Y, int VEC, int NE>
__global__ __launch_bounds__(NORM_THREADS) void gdr_norm_bwd_kernel(NormParams p, bool wide) {
    __shared__ float lds[2][4];
    const NormPlace at(p);
    if (!at.active) return;  // (never of a wide group)
    const int64_t C = (int64_t)p.groups * p.D, c0 = (int64_t)at.group * p.D;
    bool valid[NE / VEC];
    float w[NE], b[NE], dw[NE], db[NE];
#pragma unroll
    for (int v = 0; v < NE / VEC; ++v) {
        const int c = norm_channel<VEC>(v * VEC, p.lanes, at.r);
        valid[v] = c < p.D;
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            w[v * VEC + i] = 1.f;
            b[v * VEC + i] = dw[v * VEC + i] = db[v * VEC + i] = 0.f;
        }
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
        const Y *d = static_cast<const Y *>(p.dout) + t * C + c0;
        X *dx = static_cast<X *>(p.dx) + t * C + c0;
        Z *dz = static_cast<Z *>(p.dgate) + t * C + c0;
        float n[NE], a[NE], g[NE];
#pragma unroll
        for (int v = 0; v < NE / VEC; ++v) {
#pragma unroll
            for (int i = 0; i < VEC; ++i) n[v * VEC + i] = a[v * VEC + i] = g[v * VEC + i] = 0.f;
            if (!valid[v]) continue;
            const int c = norm_channel<VEC>(v * VEC, p.lanes, at.r);
            norm_load<X, VEC>(x + c, n + v * VEC);
            norm_load<Y, VEC>(d + c, g + v * VEC);
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
        float along = 0.f, mean = 0.f;
#pragma unroll
        for (int v = 0; v < NE / VEC; ++v) {
            float gz[VEC];
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                const int k = v * VEC + i;
                n[k] *= rstd;
                const float y = fmaf(n[k], w[k], b[k]);
                float slope;
                const float f = norm_act(p.act, p.gate ? a[k] : y, slope);
                gz[i] = g[k] * y * slope;
                g[k] *= p.gate ? f : slope;
                db[k] += g[k];
                dw[k] = fmaf(g[k], n[k], dw[k]);
                g[k] *= w[k];
                along = fmaf(g[k], n[k], along);
                mean += g[k];
            }
            if (p.gate && valid[v]) norm_store<Z, VEC>(dz + norm_channel<VEC>(v * VEC, p.lanes, at.r), gz);
        }
        along = sum(along) * per_channel;
        mean = p.center ? sum(mean) * per_channel : 0.f;
#pragma unroll
        for (int v = 0; v < NE / VEC; ++v) {
            if (!valid[v]) continue;
            float y[VEC];
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                const int k = v * VEC + i;
                y[i] = rstd * (fmaf(-n[k], along, g[k]) - mean);
            }
            norm_store<X, VEC>(dx + norm_channel<VEC>(v * VEC, p.lanes, at.r), y);
        }
    }
    const int64_t part = ((int64_t)blockIdx.y * at.per + at.sub) * C + c0;
#pragma unroll
    for (int v = 0; v < NE / VEC; ++v) {
        if (!valid[v]) continue;
        const int c = norm_channel<VEC>(v * VEC, p.lanes, at.r);
        if (p.part_w) norm_store<float, VEC>(p.part_w + part + c, dw + v * VEC);
        if (p.part_b) norm_store<float, VEC>(p.part_b + part + c, db + v * VEC);
    }
}

template <typename X, typename Z, typename Y, int VEC, int NE> struct Launch {
    static hipError_t go(NormGrid g, const NormParams &p, hipStream_t s) {
        launch_k(gdr_norm_bwd_kernel<X, Z, Y, VEC, NE>, dim3(g.x, g.y), dim3(NORM_THREADS), 0, s, p, p.lanes > 64);
        return hipGetLastError();
    }
};

// 32 channels, 8 threads along the parts of each
__global__ __launch_bounds__(256) void gdr_norm_sum_kernel(const float *part, float *out, int64_t parts, int64_t C) {
    __shared__ float lds[8][33];
    const int cx = threadIdx.x & 31, py = threadIdx.x >> 5;
    const int64_t c = (int64_t)blockIdx.x * 32 + cx;
    float x = 0.f;
    if (c < C)
        for (int64_t i = py; i < parts; i += 8) x += part[i * C + c];
    lds[py][cx] = x;
    __syncthreads();
    if (py == 0 && c < C) {
#pragma unroll
        for (int i = 1; i < 8; ++i) x += lds[i][cx];
        out[c] = x;
    }
}

}  // namespace

hipError_t launch_norm_bwd(Dt x, Dt gate, Dt out, NormVariant v, NormGrid g, const NormParams &p, hipStream_t s) {
    return norm_types<Launch>(x, gate, out, v, g, p, s);
}
hipError_t launch_norm_sum(const float *part, float *out, int64_t parts, int64_t C, hipStream_t s) {
    launch_k(gdr_norm_sum_kernel, dim3((uint32_t)((C + 31) / 32)), dim3(256), 0, s, part, out, parts, C);
    return hipGetLastError();
}

}  // namespace gdr
