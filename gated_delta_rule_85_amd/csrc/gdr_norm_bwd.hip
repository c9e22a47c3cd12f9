// gdr_group_norm_bwd: gradients of the group norm with its activation.
//
// With n and y as in the forward, which is computed again from x (its statistics cost no pass of
// their own: the group is in registers):
//     with a gate:  dgate = dout y act'(gate),  dy = dout act(gate);   else  dy = dout act'(y);
//     dw = sum over tokens dy n,  db = sum over tokens dy,  dn = dy w,
//     dx = rstd (dn - n mean(dn n) - mean(dn)),  the last term where the norm is centred.
// A thread keeps its channels over its tokens and their dw and db in registers; the sums of the
// workgroups are added in a second kernel.  Bound by memory: x, gate and dout read, dx and dgate written,
// once.  32768 x 8192 in bf16 (2.7 GB): 526 us, 5.1 TB/s, and 8 to 16 us for the sums.  The next token is
// not read ahead here: with the three inputs of another token a thread's registers leave room for fewer
// waves, and it took 587 us.
#include "gdr_norm.hpp"

namespace gdr {
namespace {

template <typename X, typename Z, typename Y, int VEC, int NE, bool RAGGED>
__global__ __launch_bounds__(NORM_THREADS) void gdr_norm_bwd_kernel(NormParams p, bool wide) {
    constexpr int NV = NE / VEC;
    __shared__ float lds[2][4];
    const NormPlace at(p);
    const NormChannels<VEC, NE, RAGGED> ch(p, at);
    const int64_t C = (int64_t)p.groups * p.D;
    float w[NE], b[NE], dw[NE], db[NE];
    ch.parameters(p.weight, 1.f, w);
    ch.parameters(p.bias, 0.f, b);
#pragma unroll
    for (int i = 0; i < NE; ++i) dw[i] = db[i] = 0.f;
    int turn = 0;  // two places in turn: between two writes of one lies a barrier after its reads
    auto sum = [&](float v) {
        turn ^= 1;
        return wide ? norm_sum<true>(v, p.lanes, lds[turn]) : norm_sum<false>(v, p.lanes, lds[turn]);
    };
    const float per_channel = 1.f / p.D;
    const int64_t step = (int64_t)gridDim.y * at.per;
    NormRaw<X, VEC> rx[NV] = {};
    NormRaw<Z, VEC> rz[NV] = {};
    NormRaw<Y, VEC> rd[NV] = {};
    auto fetch = [&](int64_t t) {
        ch.load(static_cast<const X *>(p.x) + t * p.x_row, rx);
        ch.load(static_cast<const Y *>(p.dout) + t * C, rd);
        if (p.gate) ch.load(static_cast<const Z *>(p.gate) + t * p.gate_row, rz);
    };
    int64_t t = (int64_t)blockIdx.y * at.per + at.sub;
    if (!at.active) t = p.M;  // (never of a wide group)
    for (; t < p.M; t += step) {
        fetch(t);
        float n[NE], a[NE], g[NE];
        ch.values(rx, n);
        ch.values(rz, a);
        ch.values(rd, g);
        X *dx = static_cast<X *>(p.dx) + t * C;
        Z *dz = static_cast<Z *>(p.dgate) + t * C;
        float total = 0.f;
        if (p.center) {
#pragma unroll
            for (int i = 0; i < NE; ++i) total += n[i];
            const float mean = sum(total) * per_channel;
#pragma unroll
            for (int i = 0; i < NE; ++i) n[i] = ch.has(i) ? n[i] - mean : 0.f;
        }
        total = 0.f;
#pragma unroll
        for (int i = 0; i < NE; ++i) total = fmaf(n[i], n[i], total);
        const float rstd = rsqrtf(fmaf(sum(total), per_channel, p.eps));
        float along = 0.f, mean = 0.f;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
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
            if (p.gate && ch.valid[v]) ch.store(dz, v, gz);
        }
        along = sum(along) * per_channel;
        mean = p.center ? sum(mean) * per_channel : 0.f;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            if (!ch.valid[v]) continue;
            float y[VEC];
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                const int k = v * VEC + i;
                y[i] = rstd * (fmaf(-n[k], along, g[k]) - mean);
            }
            ch.store(dx, v, y);
        }
    }
    if (!p.part_w && !p.part_b) return;
    // the tokens that the workgroup takes at a time
    if (at.per > 1) {
        __shared__ float sums[NORM_THREADS];
        const int places = p.groups * p.lanes;
        auto over_tokens = [&](float *x) {
#pragma unroll
            for (int i = 0; i < NE; ++i) {
                __syncthreads();
                sums[threadIdx.x] = x[i];
                __syncthreads();
                if (at.active && at.sub == 0)
                    for (int s = 1; s < at.per; ++s) x[i] += sums[threadIdx.x + s * places];
            }
        };
        over_tokens(dw);
        over_tokens(db);
        if (at.sub != 0) return;
    }
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        if (!ch.valid[v]) continue;
        if (p.part_w) ch.store(p.part_w + blockIdx.y * C, v, dw + v * VEC);
        if (p.part_b) ch.store(p.part_b + blockIdx.y * C, v, db + v * VEC);
    }
}

template <typename X, typename Z, typename Y, int VEC, int NE, bool RAGGED> struct Launch {
    static hipError_t go(NormGrid g, const NormParams &p, hipStream_t s) {
        launch_k(gdr_norm_bwd_kernel<X, Z, Y, VEC, NE, RAGGED>, dim3(g.x, g.y), dim3(NORM_THREADS), 0, s, p, p.lanes > 64);
        return hipGetLastError();
    }
};

// 16 channels, 64 threads along the parts of each, in the same order in every launch
__global__ __launch_bounds__(1024) void gdr_norm_sum_kernel(const float *part_w, const float *part_b, float *w, float *b,
                                                           int64_t parts, int64_t C) {
    __shared__ float lds[64][17];
    const float *part = blockIdx.y ? part_b : part_w;
    float *out = blockIdx.y ? b : w;
    if (!out) return;
    const int cx = threadIdx.x & 15, py = threadIdx.x >> 4;
    const int64_t c = (int64_t)blockIdx.x * 16 + cx;
    float x = 0.f;
    if (c < C) {
#pragma unroll 4
        for (int64_t i = py; i < parts; i += 64) x += part[i * C + c];
    }
    lds[py][cx] = x;
    __syncthreads();
    if (py < 4) {
#pragma unroll
        for (int i = 1; i < 16; ++i) x += lds[py + 4 * i][cx];
        lds[py][cx] = x;
    }
    __syncthreads();
    if (py == 0 && c < C) out[c] = (x + lds[1][cx]) + (lds[2][cx] + lds[3][cx]);
}

}  // namespace

hipError_t launch_norm_bwd(Dt x, Dt gate, Dt out, NormVariant v, NormGrid g, const NormParams &p, hipStream_t s) {
    return norm_types<Launch>(x, gate, out, v, g, p, s);
}
hipError_t launch_norm_sum(const float *part_w, const float *part_b, float *w, float *b, int64_t parts, int64_t C, hipStream_t s) {
    launch_k(gdr_norm_sum_kernel, dim3((uint32_t)((C + 15) / 16), 2), dim3(1024), 0, s, part_w, part_b, w, b, parts, C);
    return hipGetLastError();
}

}  // namespace gdr
