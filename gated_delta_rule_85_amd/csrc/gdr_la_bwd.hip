// What the scans of linear attention leave to do: states carried over the segments, gate
// gradients, and sums over the v heads that share a q/k head.
#include "gdr_la.hpp"

namespace gdr {
namespace {

// ------------------------------------------------------------------ la_carry
// border states from their segments' own: S_b += D_{b-1} S_{b-1} for b = 2 .. (rev: from the last
// border down, S_b += D_b S_{b+1}).  A thread takes four elements of a (sequence, head) along; what it
// reads does not wait for its sums (31 borders of 8 heads: 9.1 us in place of 12.9).
__device__ __forceinline__ void carry(const LaCarry &p, int block) {
    const int per = p.KV / 1024, unit = block / per, j = unit / p.s.Hv, hv = unit - j * p.s.Hv;
    int64_t bos, eos;
    la_bounds(p.s, j, bos, eos);
    const int64_t seg_tokens = (int64_t)p.s.seg_chunks * CH;
    const int n_seg = (int)((eos - bos + seg_tokens - 1) / seg_tokens), place = la_first(p.s, bos, j, seg_tokens);
    const int64_t first_border = la_before(p.s, bos, j, seg_tokens) + 1;
    if (n_seg < 3) return;
    const int64_t stride = (int64_t)p.s.Hv * p.KV;
    float *s = p.border + (first_border * p.s.Hv + hv) * p.KV + (block - unit * per) * 1024 + 4 * threadIdx.x;
    const float *d = p.decays + (int64_t)place * p.s.Hv + hv;
    auto at = [&](int b) { return reinterpret_cast<f32x4 *>(s + (b - 1) * stride); };
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
// (a grid of any number of (sequence, head) pairs has a bounded number of work-items)
constexpr int CARRY_WORKGROUPS = 1 << 20;
__global__ __launch_bounds__(256) void gdr_la_carry_kernel(LaCarry p) {
    const int blocks = p.s.n_seq * p.s.Hv * (p.KV / 1024);
    for (int block = blockIdx.x; block < blocks; block += gridDim.x) carry(p, block);
}

// ------------------------------------------------------------------ la_gates
// dg_t = sum over i < t <= s of what key i gives to query s.  With a_s = q_s . dq_s and
// b_i = v_i . dv_i (= k_i . dk_i), dg_t - dg_{t+1} = a_t - b_t; at a segment's first token dg is
// e^g <S, dS>, from the states on either side (0 at a sequence's start without an initial state,
// else <h0, dh0>), and behind its last one the next segment's, or <S, dht>, or 0.  The differences
// cancel from one token to the next, so that they are added in 64 bits from the far end, anew in every
// segment of 16 chunks at most; what is then missing at the near end is the sum of all errors, and
// each token gets its share of it, by the sizes of the terms: the squares of all terms from the far end to it,
// of all of the segment's (8 x 4096 tokens of 64 heads: 9.7e-7 off, without it 1.7e-6; segments of 8 chunks: 6.8e-7, and 3% longer).
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

// scale <x, y>, and the sum of its terms' squares; on every thread
__device__ __forceinline__ double2 product(const float *x, const float *y, int n, double scale, double *lds) {
    float d0 = 0.f, d1 = 0.f, v0 = 0.f, v1 = 0.f;
#pragma unroll 4
    for (int i = 4 * (int)threadIdx.x; i < n; i += 1024) {
        const f32x4 z = *reinterpret_cast<const f32x4 *>(x + i) * *reinterpret_cast<const f32x4 *>(y + i);
        d0 += z[0] + z[1], d1 += z[2] + z[3];
        v0 = fmaf(z[0], z[0], fmaf(z[1], z[1], v0)), v1 = fmaf(z[2], z[2], fmaf(z[3], z[3], v1));
    }
    return {scale * block_sum((double)d0 + d1, lds), scale * scale * block_sum((double)v0 + v1, lds)};
}

// at the first token of every segment
__global__ __launch_bounds__(256) void gdr_la_borders_kernel(LaGates p) {
    __shared__ double lds[4];
    const int place = blockIdx.x / p.s.Hv, hv = blockIdx.x - place * p.s.Hv;
    int j, m;
    if (!la_place(p.s, place, j, m)) return;
    int64_t bos, eos;
    la_bounds(p.s, j, bos, eos);
    double2 at = {0.0, 0.0};
    if (m > 0) {
        const int64_t at_border = la_before(p.s, bos, j, (int64_t)p.s.seg_chunks * CH) + m, border = (at_border * p.s.Hv + hv) * p.KV;
        const float g = p.s.g[(bos + m * (int64_t)p.s.seg_chunks * CH) * p.s.g_tok + hv];
        at = product(p.fwd + border, p.rev + border, p.KV, expf(g), lds);
    } else if (p.h0) {
        const int64_t state = ((int64_t)j * p.s.Hv + hv) * p.KV;
        if (p.dh0)
            at = product(p.h0 + state, p.dh0 + state, p.KV, 1.0, lds);
        else
            at.y = -1.0;  // not known
    }
    if (threadIdx.x == 0) p.at[blockIdx.x] = at;
}

__global__ __launch_bounds__(256) void gdr_la_gates_kernel(LaGates p) {
    __shared__ double lds[4], lds2[4];
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
    const double2 near = p.at[blockIdx.x];
    double2 far = {0.0, 0.0};
    if (hi < len)
        far = p.at[blockIdx.x + p.s.Hv];
    else if (p.last)
        for (int i = 0; i < p.n_last; ++i) {
            const double2 part = p.last[((int64_t)j * p.s.Hv + hv) * p.n_last + i];
            far.x += part.x, far.y += part.y;
        }
    // a segment's 1024 tokens at most, four per thread
    const int64_t t0 = hi - 1024 + 4 * tid, plane = (int64_t)p.s.Hv * p.tokens;
    double d[4], v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t t = t0 + i;
        d[i] = v[i] = 0.0;
        if (t >= lo) {
            const int64_t at = hv * p.tokens + bos + t;
            double a = 0.0, b = 0.0;
            for (int c = 0; c < p.n_a; ++c) a += p.a[c * plane + at];
            for (int c = 0; c < p.n_b; ++c) b += p.b[c * plane + at];
            d[i] = a - b, v[i] = a * a + b * b;
        }
    }
#pragma unroll
    for (int i = 2; i >= 0; --i) d[i] += d[i + 1], v[i] += v[i + 1];
    double after = d[0], size = v[0];  // sums from this thread on, of the wave, then of the workgroup
#pragma unroll
    for (int i = 1; i < 64; i <<= 1) {
        const double z = __shfl_down(after, i), y = __shfl_down(size, i);
        if (lane_id() + i < 64) after += z, size += y;
    }
    __syncthreads();
    if (lane_id() == 0) lds[wave_id()] = after, lds2[wave_id()] = size;
    __syncthreads();
    double rest = far.x + (after - d[0]), sizes = far.y + (size - v[0]);
    for (int i = wave_id() + 1; i < 4; ++i) rest += lds[i], sizes += lds2[i];
    const double missing = near.x - (far.x + ((lds[0] + lds[1]) + (lds[2] + lds[3])));
    const double all = near.y + far.y + ((lds2[0] + lds2[1]) + (lds2[2] + lds2[3]));
    double share = missing / all;
    if (near.y < 0.0 || !(all > 0.0) || !(fabs(share) < 1e300)) share = 0.0;
    double total = 0.0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t t = t0 + i;
        if (t < lo) continue;
        const double dg = d[i] + rest + share * (v[i] + sizes);
        if (p.s.g_tok)
            p.dg[(bos + t) * p.s.Hv + hv] = (float)dg;
        else
            total += dg;
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
// out[n] = sum over a group's heads, fp32 in the order of the heads.  Bound by memory: two heads of 128
// columns for 32768 tokens x 32 heads, 1.3 GB, in 205 us, 6.5 TB/s (part of it from the last-level cache)
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
    int64_t first = 0, end = 0;
    if (p.s.n_seq > LA_WAVE_SEQS) {
        first = p.s.cu[0], end = p.s.cu[p.s.n_seq];
    } else if (p.s.n_seq > 0) {
        const int starts = la_starts(p.s);
        first = __builtin_amdgcn_readlane(starts, 0);
        end = max(__builtin_amdgcn_readlane(starts, 63), la_offset(p.s.cu, p.s.T, p.s.n_seq));
    }
    for (int64_t i = blockIdx.x; i < first + p.s.T - end; i += gridDim.x) {
        const int64_t row = i < first ? i : end + i - first;
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (k < p.n)
                for (int64_t at = threadIdx.x; at < p.words[k]; at += 256) p.x[k][row * p.words[k] + at] = 0u;
    }
}

// ---------------------------------------------------------------- la_offsets
// One workgroup, 1024 offsets at a time (5 us for 5000)
__global__ __launch_bounds__(1024) void gdr_la_offsets_kernel(const int32_t *cu, int32_t *to, int64_t n, int64_t T) {
    __shared__ int last[2][16];  // of each wave, two turns: between two writes of one lies a barrier after its reads
    int before = 0, turn = 0;
    for (int64_t first = 0; first < n; first += 1024, turn ^= 1) {
        const int64_t i = first + threadIdx.x;
        int x = la_running_max(la_offset(cu + first, T, (int)min(n - 1 - first, (int64_t)threadIdx.x)));
        if (lane_id() == 63) last[turn][wave_id()] = x;
        __syncthreads();
        x = max(x, before);
        for (int w = 0; w < 16; ++w) {
            before = max(before, last[turn][w]);
            if (w < (int)wave_id()) x = max(x, before);
        }
        if (i < n) to[i] = x;
    }
}

}  // namespace

hipError_t launch_la_offsets(const int32_t *cu, int32_t *to, int64_t n, int64_t T, hipStream_t s) {
    launch_k(gdr_la_offsets_kernel, dim3(1), dim3(1024), 0, s, cu, to, n, T);
    return hipGetLastError();
}
hipError_t launch_la_rest(const LaRest &p, hipStream_t s) {
    launch_k(gdr_la_rest_kernel, dim3((uint32_t)(p.s.T < 1024 ? p.s.T : 1024)), dim3(256), 0, s, p);
    return hipGetLastError();
}
hipError_t launch_la_carry(const LaCarry &p, hipStream_t s) {
    const int64_t blocks = (int64_t)p.s.n_seq * p.s.Hv * (p.KV / 1024);
    launch_k(gdr_la_carry_kernel, dim3((uint32_t)(blocks < CARRY_WORKGROUPS ? blocks : CARRY_WORKGROUPS)), dim3(256), 0, s, p);
    return hipGetLastError();
}
hipError_t launch_la_gates(const LaGates &p, int items, hipStream_t s) {
    launch_k(gdr_la_borders_kernel, dim3((uint32_t)items * p.s.Hv), dim3(256), 0, s, p);
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
