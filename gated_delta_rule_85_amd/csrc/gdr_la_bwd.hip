// What the scans of linear attention leave to do: states carried over the segments, gate
// gradients, and sums over the v heads that share a q/k head.
#include "gdr_la.hpp"

namespace gdr {
namespace {

// ------------------------------------------------------------------ la_carry
// border states from their segments' own: S_b += D_{b-1} S_{b-1} for b = 2 .. (rev: from the last
// border down, S_b += D_b S_{b+1}).  A thread takes four elements of a (sequence, head) along; what it
// reads does not wait for its sums (31 borders of 8 heads: 9.1 us in place of 12.9).
__global__ __launch_bounds__(256) void gdr_la_carry_kernel(LaCarry p) {
    const int per = p.KV / 1024, unit = blockIdx.x / per, j = unit / p.s.Hv, hv = unit - j * p.s.Hv;
    int64_t bos, eos;
    la_bounds(p.s, j, bos, eos);
    const int64_t seg_tokens = (int64_t)p.s.seg_chunks * CH;
    const int n_seg = (int)((eos - bos + seg_tokens - 1) / seg_tokens), place = la_first(p.s, bos, j, seg_tokens);
    if (n_seg < 3) return;
    const int64_t stride = (int64_t)p.s.Hv * p.KV;
    float *s = p.border + ((int64_t)place * p.s.Hv + hv) * p.KV + (blockIdx.x - unit * per) * 1024 + 4 * threadIdx.x;
    const float *d = p.decays + (int64_t)place * p.s.Hv + hv;
    auto at = [&](int b) { return reinterpret_cast<f32x4 *>(s + b * stride); };
    auto border = [&](int i) { return p.rev ? n_seg - i : i; };
    f32x4 x = *at(border(1));
    constexpr int N = 8;  // borders read at a time, a group ahead of the sums
    f32x4 own[N], next[N] = {};
    float decay[N], next_decay[N] = {};
    auto fetch = [&](int first) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if (first + i >= n_seg) break;
            const int b = border(first + i);
            next[i] = *at(b), next_decay[i] = d[(int64_t)(p.rev ? b : b - 1) * p.s.Hv];
        }
    };
    fetch(2);
    for (int first = 2; first < n_seg; first += N) {
#pragma unroll
        for (int i = 0; i < N; ++i) own[i] = next[i], decay[i] = next_decay[i];
        fetch(first + N);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if (first + i >= n_seg) break;
            x = own[i] + decay[i] * x;
            *at(border(first + i)) = x;
        }
    }
}

// ------------------------------------------------------------------ la_gates
// dg_t = sum over i < t <= s of what key i gives to query s: with a_s = q_s . dq_s and
// b_i = v_i . dv_i (= k_i . dk_i), dg_t = dg at the segment's far border + sum over the segment's
// s >= t of (a_s - b_s); at the border it is e^g <S, dS>, from the states on either side.  The
// differences cancel from one token to the next, so the sums run in 64 bits and start anew at
// every border.
__device__ __forceinline__ double wave_sum(double x) {
#pragma unroll
    for (int i = 32; i; i >>= 1) x += __shfl_xor(x, i);
    return x;
}
__device__ __forceinline__ double block_sum(double x, double *lds) {  // of four waves
    x = wave_sum(x);
    __syncthreads();
    if (lane_id() == 0) lds[wave_id()] = x;
    __syncthreads();
    return lds[0] + lds[1] + lds[2] + lds[3];
}

__global__ __launch_bounds__(256) void gdr_la_gates_kernel(LaGates p) {
    __shared__ double lds[4];
    const int place = blockIdx.x / p.s.Hv, hv = blockIdx.x - place * p.s.Hv, tid = threadIdx.x;
    int j, m;
    if (!la_place(p.s, place, j, m)) {
        if (p.s.g_tok == 0 && tid == 0) p.dg[blockIdx.x] = 0.f;
        return;
    }
    int64_t bos, eos;
    la_bounds(p.s, j, bos, eos);
    const int64_t seg_tokens = (int64_t)p.s.seg_chunks * CH, len = eos - bos;
    const int64_t lo = m * seg_tokens, hi = min(len, lo + seg_tokens);
    // at the far border
    const float *x = nullptr, *y = nullptr;
    double at_border = 1.0;
    if (hi < len) {
        const int64_t border = ((int64_t)(place + 1) * p.s.Hv + hv) * p.KV;
        x = p.fwd + border, y = p.rev + border;
        const float g = p.s.g[(bos + hi) * p.s.g_tok + hv];
        at_border = expf(g);
    } else if (p.dht) {
        x = p.fwd + ((int64_t)(place - m) * p.s.Hv + hv) * p.KV, y = p.dht + ((int64_t)j * p.s.Hv + hv) * p.KV;
    }
    double carry = 0.0, total = 0.0;
    if (x) {
        float d0 = 0.f, d1 = 0.f;
        for (int i = 4 * tid; i < p.KV; i += 1024) {
            const f32x4 a = *reinterpret_cast<const f32x4 *>(x + i), b = *reinterpret_cast<const f32x4 *>(y + i);
            d0 = fmaf(a[0], b[0], fmaf(a[1], b[1], d0));
            d1 = fmaf(a[2], b[2], fmaf(a[3], b[3], d1));
        }
        carry = at_border * block_sum((double)d0 + d1, lds);
    }
    const int64_t plane = (int64_t)p.s.Hv * p.tokens;
    for (int64_t t1 = hi; t1 > lo; t1 -= 1024) {  // 1024 tokens at a time, four per thread
        const int64_t t0 = t1 - 1024 + 4 * tid;
        double d[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t t = t0 + i;
            d[i] = 0.0;
            if (t >= lo) {
                const int64_t at = hv * p.tokens + bos + t;
                for (int c = 0; c < p.n_a; ++c) d[i] += p.a[c * plane + at];
                for (int c = 0; c < p.n_b; ++c) d[i] -= p.b[c * plane + at];
            }
        }
#pragma unroll
        for (int i = 2; i >= 0; --i) d[i] += d[i + 1];
        double after = d[0];  // sums from this thread on, of the wave, then of the workgroup
#pragma unroll
        for (int i = 1; i < 64; i <<= 1) {
            const double z = __shfl_down(after, i);
            if (lane_id() + i < 64) after += z;
        }
        __syncthreads();
        if (lane_id() == 0) lds[wave_id()] = after;
        __syncthreads();
        double rest = carry + (after - d[0]);
        for (int i = wave_id() + 1; i < 4; ++i) rest += lds[i];
        carry += lds[0] + lds[1] + lds[2] + lds[3];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t t = t0 + i;
            if (t < lo) continue;
            const double dg = d[i] + rest;
            if (p.s.g_tok)
                p.dg[(bos + t) * p.s.Hv + hv] = (float)dg;
            else
                total += dg;
        }
    }
    if (p.s.g_tok == 0) {
        total = block_sum(total, lds);
        if (tid == 0) p.dg[blockIdx.x] = (float)total;
    }
}

__global__ __launch_bounds__(256) void gdr_la_sum_gates_kernel(const float *part, float *dg, int64_t places, int H) {
    __shared__ double lds[4];
    const int hv = blockIdx.x;
    double x = 0.0;
    for (int64_t i = threadIdx.x; i < places; i += 256) x += part[i * H + hv];
    x = block_sum(x, lds);
    if (threadIdx.x == 0) dg[hv] = (float)x;
}

// ------------------------------------------------------------------ la_heads
template <typename Out>
__global__ __launch_bounds__(256) void gdr_la_heads_kernel(const float *x, Out *out, int64_t n, int group, int W) {
    const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
    if (i >= n) return;
    const int64_t row = i / W;
    const float *p = x + row * group * W + (i - row * W);
    f32x4 y = __builtin_nontemporal_load(reinterpret_cast<const f32x4 *>(p));
    for (int h = 1; h < group; ++h) y += __builtin_nontemporal_load(reinterpret_cast<const f32x4 *>(p + h * W));
    if constexpr (sizeof(Out) == 4)
        *reinterpret_cast<f32x4 *>(out + i) = y;
    else
        *reinterpret_cast<bf16x4 *>(out + i) = __builtin_convertvector(y, bf16x4);
}

// ------------------------------------------------------------------ la_rest
// Rows before the first and behind the last of the packed sequences := 0.  (4 us where there are none.)
__global__ __launch_bounds__(256) void gdr_la_rest_kernel(LaRest p) {
    auto clamped = [&](int i) { return min(max((int64_t)p.cu[i], (int64_t)0), p.T); };
    const int64_t first = p.n_seq > 0 ? clamped(0) : 0, end = p.n_seq > 0 ? max(clamped(p.n_seq), first) : 0;
    for (int64_t i = blockIdx.x; i < first + p.T - end; i += gridDim.x) {
        const int64_t row = i < first ? i : end + i - first;
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (k < p.n)
                for (int64_t at = threadIdx.x; at < p.words[k]; at += 256) p.x[k][row * p.words[k] + at] = 0u;
    }
}

}  // namespace

hipError_t launch_la_rest(const LaRest &p, hipStream_t s) {
    launch_k(gdr_la_rest_kernel, dim3((uint32_t)(p.T < 1024 ? p.T : 1024)), dim3(256), 0, s, p);
    return hipGetLastError();
}
hipError_t launch_la_carry(const LaCarry &p, hipStream_t s) {
    launch_k(gdr_la_carry_kernel, dim3((uint32_t)p.s.n_seq * p.s.Hv * (p.KV / 1024)), dim3(256), 0, s, p);
    return hipGetLastError();
}
hipError_t launch_la_gates(const LaGates &p, int items, hipStream_t s) {
    launch_k(gdr_la_gates_kernel, dim3((uint32_t)items * p.s.Hv), dim3(256), 0, s, p);
    return hipGetLastError();
}
hipError_t launch_la_sum_gates(const float *part, float *dg, int64_t places, int H, hipStream_t s) {
    launch_k(gdr_la_sum_gates_kernel, dim3((uint32_t)H), dim3(256), 0, s, part, dg, places, H);
    return hipGetLastError();
}
hipError_t launch_la_heads(const float *x, void *out, Dt out_dt, int64_t tokens, int H, int group, int W, hipStream_t s) {
    const int64_t n = tokens * H * W;
    const dim3 grid((uint32_t)((n / 4 + 255) / 256));
    if (out_dt == Dt::BF16)
        launch_k(gdr_la_heads_kernel<bf16>, grid, dim3(256), 0, s, x, static_cast<bf16 *>(out), n, group, W);
    else
        launch_k(gdr_la_heads_kernel<float>, grid, dim3(256), 0, s, x, static_cast<float *>(out), n, group, W);
    return hipGetLastError();
}

}  // namespace gdr
