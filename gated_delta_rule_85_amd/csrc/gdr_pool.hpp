// Operators on a pool of recurrent states (gdr_step, gdr_la_step, gdr_tree,
// gdr_tree_accept, gdr_copy_states): parameter blocks, launchers and the lookups they share.
#pragma once

#include "gdr_kernels.hpp"
#include "gdr_lds.hpp"

namespace gdr {

struct PoolParams {
    const void *q, *k, *v;
    const float *g, *beta;
    const int32_t *cu;        // [n_seq + 1] or null
    const int32_t *slots;     // [n_seq] or null (sequence j has slot j)
    const int32_t *parents;   // [tokens] (tree, accept)
    const int32_t *accepted;  // [n_seq] (accept)
    float *states;
    void *o;
    int64_t slot_stride;                 // floats
    int64_t q_row, k_row, v_row;         // elements between a sequence's tokens
    int64_t q_batch, k_batch, v_batch;   // elements between batch rows (without cu)
    int64_t T;
    int n_seq, n_slots, Hq, Hv;
    float scale;
    int64_t g_tok;  // floats between the gates of two tokens (launch_la_step): Hv, or 0
};

struct CopyParams {
    char *dst;
    const char *src;
    const int32_t *dst_slots, *src_slots;
    int64_t dst_stride, src_stride;              // bytes between slots
    int64_t dst_layer_stride, src_layer_stride;  // bytes between layers
    int64_t slot_bytes, layers;
    int n, n_dst, n_src;
};

constexpr int TREE_MAX = 64;    // nodes of a tree
constexpr int COPY_MAX = 4096;  // entries of one copy

// tokens [bos, eos) of sequence j among [0, B T); offsets are clamped to [0, T],
// the end to the start
__device__ __forceinline__ void token_range(const PoolParams &p, int j, int64_t &bos, int64_t &eos) {
    if (p.cu) {
        bos = min(max((int64_t)p.cu[j], (int64_t)0), p.T);
        eos = min(max((int64_t)p.cu[j + 1], bos), p.T);
    } else {
        bos = (int64_t)j * p.T;
        eos = bos + p.T;
    }
}
// slot of sequence j, or -1 where it has none (a negative entry, or one past the pool)
__device__ __forceinline__ int slot_of(const PoolParams &p, int j) {
    const int s = p.slots ? p.slots[j] : j;
    return (unsigned)s < (unsigned)p.n_slots ? s : -1;
}
// element offset of row i (a token of sequence j, counted in [0, B T)) of q, k or v
__device__ __forceinline__ int64_t row_offset(const PoolParams &p, int j, int64_t i, int64_t batch, int64_t row) {
    return p.cu ? i * row : (int64_t)j * batch + (i - (int64_t)j * p.T) * row;
}
// whether an earlier sequence with tokens names the same slot; every thread of the workgroup
// calls it, for one sequence.  A wave looks through a thousand entries by itself and shares
// longer lists with the others (32768 sequences of two small heads: 757 us a step without
// sharing, 540 with it; 368 without slots to look through)
__device__ __forceinline__ bool slot_taken(const PoolParams &p, int j, int slot) {
    if (!p.slots) return false;
    __shared__ int found;
    const bool share = j >= 1024;
    if (share) {
        if (threadIdx.x == 0) found = 0;
        lds_barrier();
    }
    bool taken = false;
    const int step = share ? (int)blockDim.x : 64;
#pragma unroll 4
    for (int i = share ? (int)threadIdx.x : lane_id(); i < j; i += step) {
        int64_t b = 0, e = 1;
        if (p.cu) token_range(p, i, b, e);
        taken |= p.slots[i] == slot && e > b;
    }
    if (!share) return __ballot(taken) != 0;
    if (taken) found = 1;
    lds_barrier();
    return found != 0;
}

// Workgroup id -> head such that an XCD takes runs of 8 consecutive heads (the hardware
// deals workgroups to the 8 XCDs round robin).  A last partial run of 64 stays as dealt.
__device__ __forceinline__ int xcd_runs(int id, int nb) {
    return (id | 63) < nb ? (id & ~63) | (id & 7) << 3 | (id >> 3 & 7) : id;
}

// state values are read and written once a call
__device__ __forceinline__ f32x4 load4_once(const float *p) {
    return __builtin_nontemporal_load(reinterpret_cast<const f32x4 *>(p));
}
__device__ __forceinline__ void store4_once(float *p, f32x4 x) {
    __builtin_nontemporal_store(x, reinterpret_cast<f32x4 *>(p));
}

hipError_t launch_step(Dt dt, Dt out, int K, int V, const PoolParams &p, hipStream_t s);
hipError_t launch_la_step(Dt dt, Dt out, int K, int V, const PoolParams &p, hipStream_t s);
hipError_t launch_accept(Dt dt, int K, int V, const PoolParams &p, hipStream_t s);
// most: an upper bound on the nodes of a tree (1 .. TREE_MAX)
hipError_t launch_tree(Dt dt, Dt out, int K, int V, int most, const PoolParams &p, hipStream_t s);
hipError_t launch_copy(const CopyParams &p, hipStream_t s);

}  // namespace gdr
