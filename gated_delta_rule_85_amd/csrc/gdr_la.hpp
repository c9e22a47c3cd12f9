// Linear attention with a decay for each head (gdr_la_fwd, gdr_la_bwd): parameter blocks,
// launchers and the lookups its kernels share.
#pragma once

#include "gdr_kernels.hpp"
#include "gdr_lds.hpp"

namespace gdr {

// The sequences, their gates, and their segments of seg_chunks chunks.  Border b of a sequence
// (1 <= b < its segments) lies before token 64 seg_chunks b.  What is kept per segment of all
// sequences is indexed by la_first() + its number; there are la_slots() such places.  The states at
// the borders are indexed by la_before() + b; there are la_borders() of them.
struct LaSeqs {
    const int32_t *cu;  // [n_seq + 1] or null; of more than LA_WAVE_SEQS sequences, launch_la_offsets' table
    const float *g;
    int64_t g_tok;      // floats between the gates of two tokens (0: one gate per head)
    int64_t T;
    int n_seq, Hv, seg_chunks;
    int n_seg;          // segments of every sequence (without cu)
};

// Offsets are taken within [0, T] and as no less than any before them, so that sequences never share a
// row.  Up to 64 sequences' are held by a wave, one a lane; those of more are made into a table first.
constexpr int LA_WAVE_SEQS = 64;

// running maximum over the 64 lanes, of values of 0 or more
__device__ __forceinline__ int la_running_max(int x) {
    x = max(x, __builtin_amdgcn_update_dpp(0, x, 0x111, 0xF, 0xF, false));  // row_shr 1, 2, 4, 8: within 16 lanes
    x = max(x, __builtin_amdgcn_update_dpp(0, x, 0x112, 0xF, 0xF, false));
    x = max(x, __builtin_amdgcn_update_dpp(0, x, 0x114, 0xF, 0xF, false));
    x = max(x, __builtin_amdgcn_update_dpp(0, x, 0x118, 0xF, 0xF, false));
    x = max(x, __builtin_amdgcn_update_dpp(0, x, 0x142, 0xA, 0xF, false));  // row_bcast15, 31
    return max(x, __builtin_amdgcn_update_dpp(0, x, 0x143, 0xC, 0xF, false));
}
__device__ __forceinline__ int la_offset(const int32_t *cu, int64_t T, int i) { return min(max(cu[i], 0), (int)T); }
// offset l of lane l (n_seq <= LA_WAVE_SEQS)
__device__ __forceinline__ int la_starts(const LaSeqs &s) { return la_running_max(la_offset(s.cu, s.T, min(lane_id(), s.n_seq))); }
__device__ __forceinline__ void la_bounds(const LaSeqs &s, int starts, int j, int64_t &bos, int64_t &eos) {
    bos = __builtin_amdgcn_readlane(starts, j);
    eos = j < 63 ? __builtin_amdgcn_readlane(starts, j + 1) : max((int)bos, la_offset(s.cu, s.T, j + 1));
}
// tokens [bos, eos) of sequence j among [0, B T); of whole waves, j the same on every lane
__device__ __forceinline__ void la_bounds(const LaSeqs &s, int j, int64_t &bos, int64_t &eos) {
    if (!s.cu) {
        bos = (int64_t)j * s.T;
        eos = bos + s.T;
    } else if (s.n_seq > LA_WAVE_SEQS) {
        bos = s.cu[j], eos = s.cu[j + 1];
    } else {
        la_bounds(s, la_starts(s), __builtin_amdgcn_readfirstlane(j), bos, eos);
    }
}
// place of a sequence's first segment.  Packed: a sequence of n tokens takes n / seg_tokens + 1 places
// at most, and the sequences' places do not meet
__device__ __forceinline__ int la_first(const LaSeqs &s, int64_t bos, int j, int64_t seg_tokens) {
    return s.cu ? (int)((uint32_t)bos / (uint32_t)seg_tokens) + j : j * s.n_seg;  // (a segment has at most 2^31 tokens)
}
// place before a sequence's first border.  Packed: a sequence's borders are no more than the whole
// multiples of seg_tokens that it reaches, (bos + n) / seg_tokens - bos / seg_tokens
__device__ __forceinline__ int la_before(const LaSeqs &s, int64_t bos, int j, int64_t seg_tokens) {
    return (s.cu ? (int)((uint32_t)bos / (uint32_t)seg_tokens) : j * (s.n_seg - 1)) - 1;
}
inline int64_t la_segments(int64_t T, int64_t seg_tokens) { return T > seg_tokens ? (T + seg_tokens - 1) / seg_tokens : 1; }
inline int64_t la_slots(bool packed, int64_t T, int64_t n_seq, int64_t seg_tokens) {
    return packed ? T / seg_tokens + n_seq : n_seq * la_segments(T, seg_tokens);
}
inline int64_t la_borders(bool packed, int64_t T, int64_t n_seq, int64_t seg_tokens) {
    return packed ? T / seg_tokens : n_seq * (la_segments(T, seg_tokens) - 1);
}
// sequence and segment of a place (false: none); of whole waves.  64 sequences are looked at in a step
__device__ __forceinline__ bool la_place(const LaSeqs &s, int place, int &j, int &m) {
    const int64_t seg_tokens = (int64_t)s.seg_chunks * CH;
    if (!s.cu) {
        j = place / s.n_seg, m = place - j * s.n_seg;
        return true;
    }
    int lo = 0;  // the last sequence whose first place is not past it
    int64_t bos, eos;
    if (s.n_seq <= LA_WAVE_SEQS) {
        const int starts = la_starts(s);
        const bool before = lane_id() < s.n_seq && la_first(s, starts, lane_id(), seg_tokens) <= place;
        lo = max((int)__popcll(__ballot(before)) - 1, 0);
        la_bounds(s, starts, lo, bos, eos);
    } else {
        for (int n = s.n_seq; n > 1;) {
            const int step = (n + 63) >> 6, at = lane_id() * step;
            const bool before = at < n && la_first(s, s.cu[lo + at], lo + at, seg_tokens) <= place;
            const int skip = max((int)__popcll(__ballot(before)) - 1, 0) * step;
            lo += skip, n = min(step, n - skip);
        }
        la_bounds(s, lo, bos, eos);
    }
    j = lo;
    m = place - la_first(s, bos, lo, seg_tokens);
    return m >= 0 && (m == 0 || m * seg_tokens < eos - bos);
}

// Work of a workgroup: `share` neighbours, which read the same q and k, on one XCD's L2, and the XCDs by
// turns, since some places of packed sequences hold no segment: 32768 tokens of 8 heads in 33 places of 8
// workgroups, the last place empty, took 219 us with neighbouring places on an XCD (33 workgroups for
// the 32 compute units of seven XCDs), and 139 without it
__device__ __forceinline__ int la_work(int id, int total, int share) {
    const int k = id >> 3, turn = k / share;
    return (turn + 1) * share * 8 > total ? id : (turn * 8 + (id & 7)) * share + k % share;
}

// One scan: o_t = out_scale S_t^T q_t with S_t = e^g S + in_scale k_t v_t^T over every sequence
// and v head, S of KD x W.  The forward is one; the backward is three, with the tensors in other
// places, two of them from the last token to the first (rev: a row's gate is then the next
// token's).  q, k and v rows of v head hv are those of head hv / *_div.
struct LaJob {
    const void *q, *k, *v;
    int64_t q_row, k_row, v_row, q_batch, k_batch, v_batch;  // elements between tokens, batch rows
    int q_div, k_div, v_div;
    int rev;
    int W;                // columns of S and o, all of them
    int trans;            // states in memory are [W][KD] in place of [KD][W]
    float in_scale, out_scale;
    void *o;              // [tokens][Hv][W]
    const float *init;    // [n_seq][Hv] states, or null: zero
    float *fin;           // [n_seq][Hv] last states (rev: times e^g of the first token), or null
    float *border;        // [borders][Hv] states, or null
    const float *with;    // [n_seq][Hv] states, or null: last[n_seq][Hv][W / 16] (scale 1), a wave's part each, becomes
    double2 *last;        // the product of the last state with them and the sum of its terms' squares (dots; trans)
    float *decays;        // [places][Hv] the segments' whole decays (launch_la_states)
    // dots[cb][hv][token] = sum over the block's 64 columns of o and e (rows like o's), or null
    const void *e;
    int64_t e_row, e_batch;
    int e_div;
    float *dots;
};

struct LaParams {
    LaSeqs s;
    LaJob job[3];
    int n_jobs, n_cb;     // jobs and blocks of 64 columns in the grid
    int split;            // workgroups take a segment each, from the border states
    int share;            // neighbours in the grid that read the same q and k (launch)
    int64_t tokens;       // B T
};

// States at the borders, from a zero state (or init) at each segment's start; la_carry then adds
// what comes from before.  decays: [places][Hv] a segment's whole decay
struct LaCarry {
    LaSeqs s;
    float *border;
    const float *decays;
    int KV, rev;
};

struct LaGates {
    LaSeqs s;
    const float *fwd, *rev;  // states and their gradients at the borders
    const double2 *last;     // [n_seq][Hv][n_last] parts of <last state, dht> and of its terms' squares, or null
    int n_last;
    const float *h0, *dh0;   // [n_seq][Hv] or null
    const float *a, *b;      // [n_a | n_b][Hv][tokens] dots
    int n_a, n_b, KV;
    int64_t tokens;
    double2 *at;             // [places][Hv] dg at the segments' first tokens, and its size (see the kernel)
    float *dg;               // [tokens][Hv], or per-head partial sums [places][Hv] (s.g_tok 0)
};

// Tensors whose rows of no sequence are cleared: [T] rows of `words` 32-bit words
struct LaRest {
    LaSeqs s;
    int n;
    uint32_t *x[4];
    int64_t words[4];
};

// out: type of the jobs' o; last: the type that it is rounded to in the end; dots: whether they sum dots
hipError_t launch_la_scan(Dt dt, Dt out, Dt last, int KD, bool dots, const LaParams &p, int items, hipStream_t s);
// end states of segments only, into the border after (rev: before) each, with their decays
hipError_t launch_la_states(Dt dt, int KD, const LaParams &p, int items, hipStream_t s);
hipError_t launch_la_carry(const LaCarry &p, hipStream_t s);
hipError_t launch_la_gates(const LaGates &p, int items, hipStream_t s);
// out[token][h][d] = sum over the heads of group h of x[token][H group][W] (fp32)
hipError_t launch_la_heads(const float *x, void *out, Dt out_dt, int64_t tokens, int H, int group, int W, hipStream_t s);
hipError_t launch_la_rest(const LaRest &p, hipStream_t s);
// to[i] (n of them) = the largest of cu[0] .. cu[i], within [0, T]
hipError_t launch_la_offsets(const int32_t *cu, int32_t *to, int64_t n, int64_t T, hipStream_t s);
// dg[h] = sum over the places of part[place][h]
hipError_t launch_la_sum_gates(const float *part, float *dg, int64_t places, int H, hipStream_t s);

}  // namespace gdr
