// gdr_copy_states: states[dst[i]] = source[src[i]] for a list of entries, every
// source read before any state is written (so that lists may permute a pool in
// place), the last of the entries with the same dst standing.
//
// The bytes of a state are independent, so a workgroup takes one column (the same
// bytes of every slot) at a time and needs no scratch: it reads the column of
// every entry's source into registers, waits for all of them, and writes.
// Lane groups of LW lanes hold 16 LW bytes of one entry's column; a workgroup of NT
// threads holds RN entries per group, RN NT / LW in all.  Workgroups are persistent:
// the list is resolved once (a hash table of dst in LDS keeps the last entry of
// each), then columns are taken in turn.
//
// Bound by HBM: states read once and written once at 5.2 TB/s (61 entries of 12 layers' pools,
// 635 MB, 122 us), where a copy of 1 GB by one-to-one threads runs at 5.0; one 2 MB state
// forked to 7 slots takes 5.7 us, most of it launch and latency.
#include "gdr_pool.hpp"

namespace gdr {
namespace {

__device__ __forceinline__ uint32_t spread(uint32_t x) { return x * 2654435761u; }  // Knuth's multiplicative hash

template <int LW, int NT, int RN>
__global__ __launch_bounds__(NT) void gdr_copy_kernel(CopyParams p, int64_t columns, int bits) {
    extern __shared__ int table[];  // 1 << bits keys, then as many entries
    const int size = 1 << bits;
    int *key = table, *val = table + size;
    for (int i = threadIdx.x; i < size; i += NT) {
        key[i] = -1;
        val[i] = -1;
    }
    __syncthreads();
    constexpr int GROUPS = NT / LW;
    const int group = threadIdx.x / LW, lane = threadIdx.x % LW;
    auto valid = [&](int e, int &d, int &s) {
        if (e >= p.n) return false;
        d = p.dst_slots[e];
        s = p.src_slots[e];
        return (unsigned)d < (unsigned)p.n_dst && s < p.n_src;
    };
    // the table has at least twice as many places as there are entries, so a free or
    // equal one is always found
    for (int e = threadIdx.x; e < p.n; e += NT) {
        int d, s;
        if (!valid(e, d, s)) continue;
        uint32_t at = spread(d) >> (32 - bits);
        for (;;) {
            const int was = atomicCAS(&key[at], -1, d);
            if (was == -1 || was == d) break;
            at = (at + 1) & (size - 1);
        }
        atomicMax(&val[at], e);
    }
    __syncthreads();
    int from[RN], to[RN];  // slots of this group's entries; to < 0: none, from < 0: zeros
#pragma unroll
    for (int r = 0; r < RN; ++r) {
        const int e = r * GROUPS + group;
        int d = -1, s = -1;
        to[r] = from[r] = -1;
        if (valid(e, d, s)) {
            uint32_t at = spread(d) >> (32 - bits);
            while (key[at] != d) at = (at + 1) & (size - 1);
            if (val[at] == e) {
                to[r] = d;
                from[r] = s;
            }
        }
    }
    const int64_t width = 16 * LW, per_layer = (p.slot_bytes + width - 1) / width;
    for (int64_t c = xcd_runs(blockIdx.x, gridDim.x); c < columns; c += gridDim.x) {
        const int64_t layer = c / per_layer, at = (c - layer * per_layer) * width + 16 * lane;
        const bool inside = at < p.slot_bytes;
        const char *src = p.src + layer * p.src_layer_stride + at;
        char *dst = p.dst + layer * p.dst_layer_stride + at;
        f32x4 x[RN];
#pragma unroll
        for (int r = 0; r < RN; ++r) {
            x[r] = zero4();
            if (inside && to[r] >= 0 && from[r] >= 0)
                x[r] = *reinterpret_cast<const f32x4 *>(src + from[r] * p.src_stride);
        }
        // the values are in registers here: every load of the workgroup has returned
        // before any store to this column is issued
#pragma unroll
        for (int r = 0; r < RN; ++r) asm volatile("" : "+v"(x[r]));
        __syncthreads();
#pragma unroll
        for (int r = 0; r < RN; ++r)
            if (inside && to[r] >= 0) store4_once(reinterpret_cast<float *>(dst + to[r] * p.dst_stride), x[r]);
    }
}

template <int LW, int NT, int RN> hipError_t launch(const CopyParams &p, hipStream_t s) {
    int bits = 1;
    while ((1 << bits) < 2 * p.n) ++bits;
    const int64_t columns = p.layers * ((p.slot_bytes + 16 * LW - 1) / (16 * LW));
    // two workgroups per compute unit keep enough loads in flight where each has many;
    // with few entries, as many threads as the 256 compute units hold
    const int64_t most = 256 * (RN >= 8 ? 2 : 2048 / NT);
    const uint32_t lds = 8u << bits;
    launch_k(gdr_copy_kernel<LW, NT, RN>, dim3((uint32_t)(columns < most ? columns : most)), dim3(NT), lds, s, p, columns,
             bits);
    return hipGetLastError();
}

}  // namespace

// Few entries: wide columns, so that a slot's bytes move in runs of 1 KB.  Many: narrower
// ones, since all entries' columns are held at once.  Measured over cold pools, states read
// and written per second: 61 entries of 12 layers 5.15 TB/s with 512-byte columns and 1024
// threads (4.7 with 1 KB and 256 threads, 4.6 with 256 bytes and 512), 128 of 12 layers 5.0
// (4.6 with 256 bytes), 250 of 2 MB 4.7 (4.8); 900 of 2 MB 4.8 with 256-byte columns (4.2 with
// 128 bytes and 512 threads); 3000 of 512 KB 3.4 with 64 bytes.
hipError_t launch_copy(const CopyParams &p, hipStream_t s) {
    if (p.n <= 4) return launch<64, 256, 1>(p, s);
    if (p.n <= 16) return launch<64, 256, 4>(p, s);
    if (p.n <= 256) return launch<32, 1024, 8>(p, s);
    if (p.n <= 1024) return launch<16, 1024, 16>(p, s);
    return launch<4, 1024, 16>(p, s);  // up to COPY_MAX = 4096
}

}  // namespace gdr
