// Host side of linear attention with a decay for each head (include/gdr.h): argument
// validation, the split into segments, and the launches.
#include <algorithm>

#include "gdr_la.hpp"

using namespace gdr;

namespace {

bool aligned16(const void *p) { return ((uintptr_t)p & 15) == 0; }
int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
size_t up(size_t n) { return (n + 255) & ~(size_t)255; }

constexpr int64_t UNITS = 256;    // compute units of an MI355X, a workgroup each
constexpr int BORDER_CHUNKS = 16; // the backward's longest segments (gate gradients start anew at each border; gdr_la_gates_kernel)

// 128 columns a workgroup (bf16) where that leaves one for every compute unit (gdr_la_scan.hip): fewer
// tiles of P a column, against all compute units busy.  `units`: sequences (or segments) and heads
bool wide(int32_t dtype, int64_t units) { return dtype == GDR_BF16 && units >= UNITS; }

// Chunks per segment, or 0: no split.  N chunks a sequence, `units` sequences and heads of `blocks` times
// 64 columns, `scans` scans and `states` scans without output.  In the time of a chunk of 128 columns on every
// compute unit (4.4 us): a chunk of 64 columns takes 0.6 (backwards 0.7), one without output 0.5 of a
// workgroup that shares its compute unit; a workgroup's start 1 to 3, the launches and the carry
// between the two 3 and what the segments' states take.  Prefill of one sequence of 4096 tokens (32
// heads of 128 columns) takes 68 us split, 141 unsplit; backwards, 4 x 2048 tokens of 32 heads 421 us
// with segments of 16 and 473 unsplit.
// Of packed sequences the lengths are not known here: the time of one with all the tokens counts as much
// as that of half of them with twice the mean length.
int64_t split_chunks(int32_t dtype, int64_t N, int64_t n_seq, bool packed, int64_t heads, int64_t blocks, int64_t scans,
                     int64_t states) {
    if (N < 2) return 0;
    const double half = scans > 1 ? 0.7 : 0.6;
    auto scan = [&](int64_t u, int64_t L) {
        return blocks == 2 && wide(dtype, u) ? (double)cdiv(u, UNITS) * (L + 1) : half * (double)cdiv(u * blocks, UNITS) * (L + 1);
    };
    auto time = [&](int64_t units, int64_t n, int64_t l) {  // n chunks each, segments of l
        const int64_t S = cdiv(n, l);
        if (S < 2) return scans * scan(units, n);
        return scans * scan(S * units, l) + 0.5 * (double)cdiv(states * (S - 1) * units * blocks, 2 * UNITS) * (l + 3) + 3 + S / 16.0;
    };
    auto all = [&](int64_t l) {
        return packed ? time(heads, N, l) + time(cdiv(n_seq, 2) * heads, cdiv(2 * N, n_seq + 1), l) : time(n_seq * heads, N, l);
    };
    const int64_t units = packed ? heads : n_seq * heads;
    double best = all(N);
    int64_t L = 0;
    for (int64_t S = 2; S <= N && (S - 1) * units < 4 * UNITS; ++S) {
        const int64_t l = cdiv(N, S);
        if (cdiv(N, l) != S) continue;  // the segments of a smaller S
        const double t = all(l);
        if (t < best) best = t, L = l;
    }
    return L;
}

template <typename Args> int check(const Args *a, int32_t out_dtype) {
    if (!a || a->B < 0 || a->T < 0 || a->H_q < 1 || a->H_v < 1 || a->H_v % a->H_q != 0) return GDR_EINVAL;
    const bool varlen = a->cu_seqlens != nullptr;
    if (varlen && (a->B != 1 || a->n_seq < 0)) return GDR_EINVAL;
    if (a->dtype != GDR_BF16 && a->dtype != GDR_F32) return GDR_ENOTSUP;
    if (out_dtype != GDR_BF16 && out_dtype != GDR_F32) return GDR_ENOTSUP;
    if ((a->K != 64 && a->K != 128) || (a->V != 64 && a->V != 128)) return GDR_ENOTSUP;
    const int64_t limit = ((int64_t)1 << 31) - 64, n_seq = varlen ? a->n_seq : a->B;
    if (a->segment_chunks < 0 || a->T >= limit || n_seq >= limit || a->H_v >= 65536) return GDR_EINVAL;
    if (a->T > 0 && a->B >= cdiv(limit, a->T)) return GDR_EINVAL;
    const int64_t per16 = a->dtype == GDR_BF16 ? 8 : 4;
    for (const int64_t st : {a->q_row, a->k_row, a->v_row})
        if (st < 0 || st % per16 != 0 || st >= 1 << 23) return GDR_EINVAL;  // 64 rows within 32-bit byte offsets
    if (!varlen)
        for (const int64_t st : {a->q_batch, a->k_batch, a->v_batch})
            if (st < 0 || st % per16 != 0) return GDR_EINVAL;
    if (!aligned16(a->q) || !aligned16(a->k) || !aligned16(a->v) || !aligned16(a->initial_state)) return GDR_EINVAL;
    return GDR_OK;
}

// Sequences and segments, and where the borders' states lie
struct Plan {
    int64_t n_seq, tokens, seg_tokens, places;
    int group, n_cb_k, n_cb_v;  // blocks of columns, where K or V columns are scanned
    bool split;
    int seg_chunks;
    size_t offsets_bytes, off_offsets, border_bytes, decays_bytes, off_fwd, off_rev, off_decays_fwd, off_decays_rev, off_dots, off_dq, off_dk, off_gates, off_at, off_last, total;
};

template <typename Args> int plan(const Args *a, bool backward, Plan &p) {
    const bool varlen = a->cu_seqlens != nullptr;
    p.n_seq = varlen ? a->n_seq : a->B;
    p.tokens = p.n_seq > 0 ? a->B * a->T : 0;
    p.group = (int)(a->H_v / a->H_q);
    const int64_t nct = cdiv(a->T, CH);
    int64_t L = a->segment_chunks ? a->segment_chunks
                                  : split_chunks(a->dtype, nct, std::max<int64_t>(p.n_seq, 1), varlen, a->H_v,
                                                 std::max(a->V, backward ? a->K : 0) / 64, backward ? 3 : 1, backward ? 2 : 1);
    const int64_t limit = (int64_t)1 << 22;  // (sequence or segment, v head) pairs
    p.split = L > 0 && L < nct;
    if (backward) L = L > 0 ? std::min<int64_t>(L, BORDER_CHUNKS) : BORDER_CHUNKS;
    // (no split of its own accord into too many)
    if (p.split && !a->segment_chunks && la_slots(varlen, a->T, p.n_seq, L * CH) * a->H_v >= limit) p.split = false;
    if (!p.split && !backward) L = std::max<int64_t>(nct, 1);
    p.seg_chunks = (int)L;
    p.seg_tokens = L * CH;
    p.places = la_slots(varlen, a->T, p.n_seq, p.seg_tokens);
    // 32-bit numbers of work-items: 1024 at most per pair, 256 of the backward's borders where there is no split
    if ((p.split ? p.places : p.n_seq) * a->H_v >= limit || p.places * a->H_v >= 4 * limit) return GDR_EINVAL;
    const bool whole = wide(a->dtype, (p.split ? p.places : p.n_seq) * a->H_v);
    p.n_cb_k = a->K == 128 && !whole ? 2 : 1, p.n_cb_v = a->V == 128 && !whole ? 2 : 1;
    p.border_bytes = up(sizeof(float) * (size_t)(la_borders(varlen, a->T, p.n_seq, p.seg_tokens) * a->H_v * a->K * a->V));
    p.decays_bytes = up(sizeof(float) * (size_t)(p.places * a->H_v));
    p.offsets_bytes = varlen && p.n_seq > LA_WAVE_SEQS ? up(sizeof(int32_t) * (size_t)(p.n_seq + 1)) : 0;
    return GDR_OK;
}

int plan_fwd(const gdr_la_fwd_args *a, Plan &p) {
    int rc = a ? check(a, a->out_dtype) : GDR_EINVAL;
    if (rc) return rc;
    rc = plan(a, false, p);
    if (rc) return rc;
    p.off_fwd = 0;
    p.off_decays_fwd = p.border_bytes;
    p.off_offsets = p.split ? p.border_bytes + p.decays_bytes : 0;
    p.total = p.off_offsets + p.offsets_bytes;
    return GDR_OK;
}

int plan_bwd(const gdr_la_bwd_args *a, Plan &p) {
    int rc = a ? check(a, a->grad_dtype) : GDR_EINVAL;
    if (rc) return rc;
    rc = plan(a, true, p);
    if (rc) return rc;
    if (p.group > 1 && p.tokens * a->H_q * a->K >= (int64_t)1 << 34) return GDR_EINVAL;  // work-items of the sums
    size_t off = 0;
    auto take = [&](size_t n) {
        const size_t at = off;
        off += up(n);
        return at;
    };
    p.off_fwd = take(p.border_bytes), p.off_rev = take(p.border_bytes);
    p.off_decays_fwd = take(p.decays_bytes), p.off_decays_rev = take(p.decays_bytes);
    const size_t tokens = (size_t)p.tokens * a->H_v * sizeof(float);
    p.off_dots = take(tokens * (p.n_cb_k + p.n_cb_v));
    p.off_dq = take(p.group > 1 ? tokens * a->K : 0), p.off_dk = take(p.group > 1 ? tokens * a->K : 0);
    p.off_gates = take(p.decays_bytes);
    p.off_at = take(4 * p.decays_bytes);
    p.off_last = take(sizeof(double2) * (size_t)(p.n_seq * a->H_v * (a->K / 16)));
    p.off_offsets = take(p.offsets_bytes);
    p.total = off;
    return GDR_OK;
}

int64_t words(int64_t elements, int32_t t) { return t == GDR_BF16 ? elements / 2 : elements; }

Dt type_of(int32_t t) { return t == GDR_BF16 ? Dt::BF16 : Dt::F32; }

template <typename Args> LaSeqs sequences(const Args *a, const Plan &p) {
    const int32_t *cu = p.offsets_bytes ? reinterpret_cast<const int32_t *>(static_cast<const char *>(a->workspace) + p.off_offsets) : a->cu_seqlens;
    return {cu, a->g, a->g_per_head ? 0 : a->H_v, a->T, (int)p.n_seq, (int)a->H_v, p.seg_chunks,
            (int)la_segments(a->T, p.seg_tokens)};
}

// the table that `s` has for its offsets, where it has one
template <typename Args> hipError_t make_offsets(const Args *a, const Plan &p, const LaSeqs &s, hipStream_t stream) {
    return p.offsets_bytes ? launch_la_offsets(a->cu_seqlens, const_cast<int32_t *>(s.cu), p.n_seq + 1, a->T, stream) : hipSuccess;
}

// neighbours of a grid: the v heads, blocks of columns and jobs of a q/k head
int neighbours(const Plan &p, const LaParams &l) { return std::min(p.group * l.n_cb * l.n_jobs, 8); }

// launches bind to the timing stage open on this thread (launch_k): none is
struct NoStage {
    NoStage() { stage_events() = {nullptr, nullptr, false}; }
    ~NoStage() { stage_events() = {nullptr, nullptr, false}; }
};

}  // namespace

extern "C" {

int gdr_la_fwd_workspace(const gdr_la_fwd_args *a, size_t *bytes) {
    if (!bytes) return GDR_EINVAL;
    Plan p;
    const int rc = plan_fwd(a, p);
    if (!rc) *bytes = p.total;
    return rc;
}

int gdr_la_bwd_workspace(const gdr_la_bwd_args *a, size_t *bytes) {
    if (!bytes) return GDR_EINVAL;
    Plan p;
    const int rc = plan_bwd(a, p);
    if (!rc) *bytes = p.total;
    return rc;
}

int gdr_la_fwd(const gdr_la_fwd_args *a, hipStream_t stream) {
    Plan pl;
    const int rc = plan_fwd(a, pl);
    if (rc) return rc;
    const bool rest = a->zero_rest && a->cu_seqlens && a->T > 0;
    if (rest && !a->o) return GDR_EINVAL;
    if (!rest && (pl.n_seq == 0 || (pl.tokens == 0 && !a->final_state))) return GDR_OK;
    if (pl.tokens > 0 && (!a->q || !a->k || !a->v || !a->g || !a->o)) return GDR_EINVAL;
    if (!aligned16(a->o) || !aligned16(a->final_state) || !aligned16(a->workspace)) return GDR_EINVAL;
    if (pl.total > 0 && (!a->workspace || a->workspace_bytes < pl.total)) return GDR_EWORKSPACE;
    const NoStage stage;
    const LaSeqs s = sequences(a, pl);
    if (make_offsets(a, pl, s, stream) != hipSuccess) return GDR_ELAUNCH;
    if (rest) {
        const LaRest r = {s, 1, {static_cast<uint32_t *>(a->o)}, {words(a->H_v * a->V, a->out_dtype)}};
        if (launch_la_rest(r, stream) != hipSuccess) return GDR_ELAUNCH;
        if (pl.n_seq == 0) return GDR_OK;
    }
    char *ws = static_cast<char *>(a->workspace);
    float *border = pl.split ? reinterpret_cast<float *>(ws + pl.off_fwd) : nullptr;
    LaParams p = {};
    p.s = s;
    p.n_jobs = 1, p.n_cb = pl.n_cb_v, p.split = pl.split, p.tokens = pl.tokens;
    LaJob &J = p.job[0];
    J.q = a->q, J.k = a->k, J.v = a->v;
    J.q_row = a->q_row, J.k_row = a->k_row, J.v_row = a->v_row;
    J.q_batch = a->q_batch, J.k_batch = a->k_batch, J.v_batch = a->v_batch;
    J.q_div = J.k_div = pl.group, J.v_div = 1;
    J.W = (int)a->V, J.in_scale = 1.f, J.out_scale = a->scale;
    J.o = a->o;
    J.init = a->initial_state, J.fin = a->final_state, J.border = border;
    const Dt dt = type_of(a->dtype);
    if (pl.split) {
        J.decays = reinterpret_cast<float *>(ws + pl.off_decays_fwd);
        p.n_cb = (int)(a->V / 64), p.share = neighbours(pl, p);
        if (launch_la_states(dt, (int)a->K, p, (int)pl.places, stream) != hipSuccess) return GDR_ELAUNCH;
        const LaCarry c = {p.s, border, J.decays, (int)(a->K * a->V), 0};
        if (launch_la_carry(c, stream) != hipSuccess) return GDR_ELAUNCH;
        p.n_cb = pl.n_cb_v;
    }
    p.share = neighbours(pl, p);
    const int items = (int)(pl.split ? pl.places : pl.n_seq);
    return launch_la_scan(dt, type_of(a->out_dtype), type_of(a->out_dtype), (int)a->K, false, p, items, stream) == hipSuccess ? GDR_OK : GDR_ELAUNCH;
}

int gdr_la_bwd(const gdr_la_bwd_args *a, hipStream_t stream) {
    Plan pl;
    const int rc = plan_bwd(a, pl);
    if (rc) return rc;
    const bool rest = a->zero_rest && a->cu_seqlens && a->T > 0;
    if (rest && (!a->dq || !a->dk || !a->dv || !a->dg)) return GDR_EINVAL;
    if (pl.n_seq == 0 && !a->g_per_head && !rest) return GDR_OK;
    if (((pl.tokens > 0 || a->g_per_head) && !a->dg) || !aligned16(a->workspace)) return GDR_EINVAL;
    if (pl.tokens > 0 && (!a->q || !a->k || !a->v || !a->g || !a->dout || !a->dq || !a->dk || !a->dv)) return GDR_EINVAL;
    for (const void *x : {(const void *)a->dout, (const void *)a->dht, (const void *)a->dq, (const void *)a->dk, (const void *)a->dv,
                          (const void *)a->dh0})
        if (!aligned16(x)) return GDR_EINVAL;
    if (pl.total > 0 && (!a->workspace || a->workspace_bytes < pl.total)) return GDR_EWORKSPACE;
    const NoStage stage;
    char *ws = static_cast<char *>(a->workspace);
    auto at = [&](size_t off) { return reinterpret_cast<float *>(ws + off); };
    const Dt dt = type_of(a->dtype), gt = type_of(a->grad_dtype);
    const int K = (int)a->K, V = (int)a->V, H = (int)a->H_v, group = pl.group, items = (int)(pl.split ? pl.places : pl.n_seq);
    const int64_t do_row = (int64_t)H * V, do_batch = a->T * do_row;
    float *border_fwd = at(pl.off_fwd), *border_rev = at(pl.off_rev), *decays_fwd = at(pl.off_decays_fwd), *decays_rev = at(pl.off_decays_rev);
    float *dots_a = at(pl.off_dots), *dots_b = dots_a + (int64_t)pl.n_cb_k * H * pl.tokens;
    const LaSeqs s = sequences(a, pl);
    if (make_offsets(a, pl, s, stream) != hipSuccess) return GDR_ELAUNCH;

    // the backward's scans: dq forwards over S^T, dv backwards over dS, dk backwards over dS^T
    LaJob dq = {}, dv = {}, dk = {};
    dq.q = a->dout, dq.q_row = do_row, dq.q_batch = do_batch, dq.q_div = 1;
    dq.k = a->v, dq.k_row = a->v_row, dq.k_batch = a->v_batch, dq.k_div = 1;
    dq.v = a->k, dq.v_row = a->k_row, dq.v_batch = a->k_batch, dq.v_div = group;
    dq.e = a->q, dq.e_row = a->q_row, dq.e_batch = a->q_batch, dq.e_div = group, dq.dots = dots_a;
    dq.W = K, dq.trans = 1, dq.in_scale = 1.f, dq.out_scale = a->scale;
    dq.init = a->initial_state, dq.border = border_fwd;
    dq.with = a->dht, dq.last = reinterpret_cast<double2 *>(ws + pl.off_last);

    dv.q = a->k, dv.q_row = a->k_row, dv.q_batch = a->k_batch, dv.q_div = group;
    dv.k = a->q, dv.k_row = a->q_row, dv.k_batch = a->q_batch, dv.k_div = group;
    dv.v = a->dout, dv.v_row = do_row, dv.v_batch = do_batch, dv.v_div = 1;
    dv.e = a->v, dv.e_row = a->v_row, dv.e_batch = a->v_batch, dv.e_div = 1, dv.dots = dots_b;
    dv.W = V, dv.rev = 1, dv.in_scale = a->scale, dv.out_scale = 1.f;
    dv.init = a->dht, dv.fin = a->dh0, dv.border = border_rev;
    dv.o = a->dv;

    dk.q = a->v, dk.q_row = a->v_row, dk.q_batch = a->v_batch, dk.q_div = 1;
    dk.k = a->dout, dk.k_row = do_row, dk.k_batch = do_batch, dk.k_div = 1;
    dk.v = a->q, dk.v_row = a->q_row, dk.v_batch = a->q_batch, dk.v_div = group;
    dk.W = K, dk.rev = 1, dk.trans = 1, dk.in_scale = a->scale, dk.out_scale = 1.f;
    dk.init = a->dht, dk.border = pl.split ? border_rev : nullptr;

    // of several v heads: per head, summed afterwards
    const Dt qt = group > 1 ? Dt::F32 : gt;
    dq.o = group > 1 ? at(pl.off_dq) : a->dq, dk.o = group > 1 ? at(pl.off_dk) : a->dk;

    if (pl.n_seq > 0) {
        if (pl.split) {
            LaParams p = {};
            p.s = s, p.n_jobs = 2, p.n_cb = V / 64, p.split = 1, p.tokens = pl.tokens;
            LaJob &f = p.job[0], &r = p.job[1];
            f.k = a->k, f.k_row = a->k_row, f.k_batch = a->k_batch, f.k_div = group;
            f.v = a->v, f.v_row = a->v_row, f.v_batch = a->v_batch, f.v_div = 1;
            f.q_div = f.e_div = 1;
            f.W = V, f.in_scale = 1.f, f.init = a->initial_state, f.border = border_fwd, f.decays = decays_fwd;
            r = dv;
            r.decays = decays_rev;
            p.share = neighbours(pl, p);
            if (launch_la_states(dt, K, p, items, stream) != hipSuccess) return GDR_ELAUNCH;
            LaCarry c = {s, border_fwd, decays_fwd, K * V, 0};
            if (launch_la_carry(c, stream) != hipSuccess) return GDR_ELAUNCH;
            c = {s, border_rev, decays_rev, K * V, 1};
            if (launch_la_carry(c, stream) != hipSuccess) return GDR_ELAUNCH;
        }
        LaParams p = {};
        p.s = s, p.split = pl.split, p.tokens = pl.tokens;
        p.n_jobs = 1, p.n_cb = pl.n_cb_k, p.share = neighbours(pl, p);
        p.job[0] = dq;
        if (launch_la_scan(dt, qt, gt, V, true, p, items, stream) != hipSuccess) return GDR_ELAUNCH;
        p.job[0] = dk;
        if (launch_la_scan(dt, qt, gt, V, false, p, items, stream) != hipSuccess) return GDR_ELAUNCH;
        p.n_cb = pl.n_cb_v, p.share = neighbours(pl, p);
        p.job[0] = dv;
        if (launch_la_scan(dt, gt, gt, K, true, p, items, stream) != hipSuccess) return GDR_ELAUNCH;
        if (group > 1 && pl.tokens > 0) {
            if (launch_la_heads(static_cast<float *>(dq.o), a->dq, gt, pl.tokens, (int)a->H_q, group, K, stream) != hipSuccess) return GDR_ELAUNCH;
            if (launch_la_heads(static_cast<float *>(dk.o), a->dk, gt, pl.tokens, (int)a->H_q, group, K, stream) != hipSuccess) return GDR_ELAUNCH;
        }
        LaGates g = {s, border_fwd, border_rev, a->dht ? dq.last : nullptr, K / 16, a->initial_state, a->dh0, dots_a, dots_b, pl.n_cb_k, pl.n_cb_v, K * V, pl.tokens,
                     reinterpret_cast<double2 *>(ws + pl.off_at), a->g_per_head ? at(pl.off_gates) : a->dg};
        if (launch_la_gates(g, (int)pl.places, stream) != hipSuccess) return GDR_ELAUNCH;
    }
    if (rest) {  // (after the sums over the heads, which are made of every row)
        const int64_t qk = words(a->H_q * a->K, a->grad_dtype);
        const LaRest r = {s, a->g_per_head ? 3 : 4,
                          {static_cast<uint32_t *>(a->dq), static_cast<uint32_t *>(a->dk), static_cast<uint32_t *>(a->dv), reinterpret_cast<uint32_t *>(a->dg)},
                          {qk, qk, words(a->H_v * a->V, a->grad_dtype), a->H_v}};
        if (launch_la_rest(r, stream) != hipSuccess) return GDR_ELAUNCH;
    }
    if (a->g_per_head && launch_la_sum_gates(at(pl.off_gates), a->dg, pl.n_seq > 0 ? pl.places : 0, H, stream) != hipSuccess)
        return GDR_ELAUNCH;
    return GDR_OK;
}

}  // extern "C"
