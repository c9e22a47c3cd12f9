// gdr_tree: the gated delta rule for a tree of drafted tokens over a cached state.
//
// Node i of a tree has the state that the recurrence reaches over the nodes on
// its path; node j is on it if j is an ancestor of i.  With G_i the sum of g over
// the path to i, and D_ij = e^(G_i - G_j) for ancestors j of i, the corrected
// values and the outputs are those of the chunked form with the tree's mask:
//     u_i = beta_i (v_i - e^G_i k_i h - sum_j D_ij (k_i . k_j) u_j)
//     o_i = scale (e^G_i q_i h + sum_j D_ij (q_i . k_j) u_j + (q_i . k_i) u_i)
// A parent comes before its children, so that one pass in node order solves for u.
#include "gdr_pool.hpp"

namespace gdr {
namespace {

template <typename In, typename Out, int K>
__global__ __launch_bounds__(128) void gdr_tree_kernel(PoolParams p, int V) {
    __shared__ float ks[TREE_MAX][K], qs[TREE_MAX][K];
    __shared__ double G[TREE_MAX];
    __shared__ uint64_t mask[TREE_MAX];
    const int unit = blockIdx.x, j = unit / p.Hv, hv = unit - j * p.Hv, hq = hv / (p.Hv / p.Hq);
    const int col = threadIdx.x;
    int64_t bos, eos;
    token_range(p, j, bos, eos);
    const int64_t len = eos - bos;
    if (len <= 0) return;
    const int slot = slot_of(p, j);
    Out *o = reinterpret_cast<Out *>(p.o) + hv * V + col;
    if (slot < 0 || len > TREE_MAX) {
        for (int64_t i = bos; i < eos; ++i) o[i * p.Hv * V] = (Out)(slot < 0 ? 0.f : __builtin_nanf(""));
        return;
    }
    const int n = (int)len;
    const In *kp = reinterpret_cast<const In *>(p.k) + hq * K, *qp = reinterpret_cast<const In *>(p.q) + hq * K;
    for (int i = 0; i < n; ++i)
        for (int d = threadIdx.x; d < K; d += blockDim.x) {
            ks[i][d] = to_f32(kp[row_offset(p, j, bos + i, p.k_batch, p.k_row) + d]);
            qs[i][d] = to_f32(qp[row_offset(p, j, bos + i, p.q_batch, p.q_row) + d]);
        }
    if (threadIdx.x == 0)
        for (int i = 0; i < n; ++i) {
            const int up = p.parents[bos + i];
            const bool child = up >= 0 && up < i;
            mask[i] = child ? mask[up] | 1ull << up : 0;
            // e^g below 2^-149 is zero: a floor keeps differences of sums finite
            const float g = p.g[(bos + i) * p.Hv + hv];
            G[i] = (child ? G[up] : 0.0) + (double)(g < -200.f ? -200.f : g);
        }
    __syncthreads();
    const float *h = p.states + (int64_t)slot * p.slot_stride + (int64_t)hv * K * V + col;
    const In *vp = reinterpret_cast<const In *>(p.v) + hv * V + col;
    float u[TREE_MAX];
    for (int i = 0; i < n; ++i) {
        float kh = 0.f, qh = 0.f, qk = 0.f;
        for (int d = 0; d < K; ++d) {
            const float x = h[d * V];
            kh += ks[i][d] * x;
            qh += qs[i][d] * x;
            qk += ks[i][d] * qs[i][d];
        }
        const float eg = expf((float)G[i]);
        float su = 0.f, so = 0.f;
        for (uint64_t m = mask[i]; m; m &= m - 1) {
            const int a = __builtin_ctzll(m);
            float kk = 0.f, qa = 0.f;
            for (int d = 0; d < K; ++d) {
                kk += ks[i][d] * ks[a][d];
                qa += qs[i][d] * ks[a][d];
            }
            const float w = expf((float)(G[i] - G[a])) * u[a];
            su += kk * w;
            so += qa * w;
        }
        const float beta = p.beta[(bos + i) * p.Hv + hv];
        u[i] = beta * (to_f32(vp[row_offset(p, j, bos + i, p.v_batch, p.v_row)]) - eg * kh - su);
        o[(bos + i) * p.Hv * V] = (Out)(p.scale * (eg * qh + so + qk * u[i]));
    }
}

template <typename In, typename Out>
hipError_t launch(int K, int V, const PoolParams &p, hipStream_t s) {
    const dim3 grid((uint32_t)p.n_seq * p.Hv);
    if (K == 128)
        launch_k(gdr_tree_kernel<In, Out, 128>, grid, dim3(V), 0, s, p, V);
    else
        launch_k(gdr_tree_kernel<In, Out, 64>, grid, dim3(V), 0, s, p, V);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_tree(Dt dt, Dt out, int K, int V, int most, const PoolParams &p, hipStream_t s) {
    (void)most;
    if (dt == Dt::BF16) return out == Dt::BF16 ? launch<bf16, bf16>(K, V, p, s) : launch<bf16, float>(K, V, p, s);
    return out == Dt::BF16 ? launch<float, bf16>(K, V, p, s) : launch<float, float>(K, V, p, s);
}

}  // namespace gdr
