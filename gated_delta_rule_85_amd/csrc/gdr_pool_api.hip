// Host side of the operators on a pool of states (include/gdr.h): argument
// validation and launches.
#include "gdr_pool.hpp"

using namespace gdr;

static_assert(TREE_MAX == GDR_TREE_MAX && COPY_MAX == GDR_COPY_MAX, "limits of include/gdr.h");

namespace {

bool aligned16(const void *p) { return ((uintptr_t)p & 15) == 0; }

enum class Op { STEP, TREE, ACCEPT, LA_STEP };

// fills p; `idle`: there is nothing to launch
int plan(const gdr_pool_args *a, Op op, PoolParams &p, bool &idle) {
    if (!a || a->B < 0 || a->T < 0 || a->H_q < 1 || a->H_v < 1 || a->H_v % a->H_q != 0) return GDR_EINVAL;
    const bool varlen = a->cu_seqlens != nullptr;
    if (varlen && (a->B != 1 || a->n_seq < 0)) return GDR_EINVAL;
    if (a->dtype != GDR_BF16 && a->dtype != GDR_F32) return GDR_ENOTSUP;
    if (op != Op::ACCEPT && a->out_dtype != GDR_BF16 && a->out_dtype != GDR_F32) return GDR_ENOTSUP;
    if ((a->K != 64 && a->K != 128) || (a->V != 64 && a->V != 128)) return GDR_ENOTSUP;
    const int64_t n_seq = varlen ? a->n_seq : a->B, limit = (int64_t)1 << 31;
    // 32-bit sequence and head numbers, and one workgroup per (sequence, v head)
    if (a->T >= limit || n_seq >= limit || a->H_v >= limit || n_seq * a->H_v > (int64_t)1 << 22) return GDR_EINVAL;
    if (a->B * a->T >= limit) return GDR_EINVAL;
    const bool steps = op == Op::STEP || op == Op::LA_STEP;
    if (!steps && !varlen && a->T > GDR_TREE_MAX) return GDR_EINVAL;
    if (a->n_slots < 1 || a->n_slots >= limit || (!a->slots && a->n_slots < n_seq)) return GDR_EINVAL;
    if (a->n_slots > 1 && (a->slot_stride % 4 != 0 || a->slot_stride < a->H_v * a->K * a->V)) return GDR_EINVAL;
    const int64_t per16 = a->dtype == GDR_BF16 ? 8 : 4;
    for (const int64_t st : {a->k_row, a->v_row, op == Op::ACCEPT ? 0 : a->q_row, varlen ? 0 : a->k_batch,
                             varlen ? 0 : a->v_batch, varlen || op == Op::ACCEPT ? 0 : a->q_batch})
        if (st < 0 || st % per16 != 0) return GDR_EINVAL;
    // 64 rows of a tree lie within 32-bit byte offsets
    if (a->H_v >= 65536 || a->k_row >= 1 << 23 || a->v_row >= 1 << 23 || (op != Op::ACCEPT && a->q_row >= 1 << 23))
        return GDR_EINVAL;
    idle = n_seq == 0 || a->T == 0;
    if (idle) return GDR_OK;
    if (!a->k || !a->v || !a->g || (op != Op::LA_STEP && !a->beta) || !a->states) return GDR_EINVAL;
    if (op != Op::ACCEPT && (!a->q || !a->o)) return GDR_EINVAL;
    if (!steps && !a->parents) return GDR_EINVAL;
    if (op == Op::ACCEPT && !a->accepted) return GDR_EINVAL;
    if (!aligned16(a->k) || !aligned16(a->v) || !aligned16(a->states)) return GDR_EINVAL;
    if (op != Op::ACCEPT && (!aligned16(a->q) || !aligned16(a->o))) return GDR_EINVAL;
    p = {a->q, a->k, a->v, a->g, a->beta, a->cu_seqlens, a->slots, a->parents, a->accepted, a->states, a->o,
         a->n_slots > 1 ? a->slot_stride : 0, a->q_row, a->k_row, a->v_row, a->q_batch, a->k_batch, a->v_batch,
         a->T, (int)n_seq, (int)a->n_slots, (int)a->H_q, (int)a->H_v, a->scale,
         op == Op::LA_STEP && a->g_per_head ? 0 : a->H_v};
    return GDR_OK;
}

Dt type_of(int32_t t) { return t == GDR_BF16 ? Dt::BF16 : Dt::F32; }

// launches bind to the timing stage open on this thread (launch_k): none is
int done(hipError_t e) {
    stage_events() = {nullptr, nullptr, false};
    return e == hipSuccess ? GDR_OK : GDR_ELAUNCH;
}

}  // namespace

extern "C" {

int gdr_step(const gdr_pool_args *a, hipStream_t stream) {
    PoolParams p;
    bool idle = false;
    const int rc = plan(a, Op::STEP, p, idle);
    if (rc || idle) return rc;
    return done(launch_step(type_of(a->dtype), type_of(a->out_dtype), (int)a->K, (int)a->V, p, stream));
}

int gdr_la_step(const gdr_pool_args *a, hipStream_t stream) {
    PoolParams p;
    bool idle = false;
    const int rc = plan(a, Op::LA_STEP, p, idle);
    if (rc || idle) return rc;
    return done(launch_la_step(type_of(a->dtype), type_of(a->out_dtype), (int)a->K, (int)a->V, p, stream));
}

int gdr_tree(const gdr_pool_args *a, hipStream_t stream) {
    PoolParams p;
    bool idle = false;
    const int rc = plan(a, Op::TREE, p, idle);
    if (rc || idle) return rc;
    const int most = (int)(a->T < GDR_TREE_MAX ? a->T : GDR_TREE_MAX);
    return done(launch_tree(type_of(a->dtype), type_of(a->out_dtype), (int)a->K, (int)a->V, most, p, stream));
}

int gdr_tree_accept(const gdr_pool_args *a, hipStream_t stream) {
    PoolParams p;
    bool idle = false;
    const int rc = plan(a, Op::ACCEPT, p, idle);
    if (rc || idle) return rc;
    return done(launch_accept(type_of(a->dtype), (int)a->K, (int)a->V, p, stream));
}

int gdr_copy_states(const gdr_copy_args *a, hipStream_t stream) {
    const int64_t limit = (int64_t)1 << 31;
    if (!a || a->n < 0 || a->n > GDR_COPY_MAX || a->layers < 0 || a->slot_bytes < 0 || a->slot_bytes % 16 != 0)
        return GDR_EINVAL;
    if (a->n_dst < 1 || a->n_dst >= limit || a->n_src < 1 || a->n_src >= limit) return GDR_EINVAL;
    if (a->n_dst > 1 && (a->dst_stride % 16 != 0 || a->dst_stride < a->slot_bytes)) return GDR_EINVAL;
    if (a->n_src > 1 && (a->src_stride % 16 != 0 || a->src_stride < a->slot_bytes)) return GDR_EINVAL;
    if (a->dst_layer_stride % 16 != 0 || a->dst_layer_stride < 0) return GDR_EINVAL;
    if (a->src_layer_stride % 16 != 0 || a->src_layer_stride < 0) return GDR_EINVAL;
    // states that share memory would be written twice: the slots of one layer lie apart from
    // the next layer's, or the layers of one slot apart from the next slot's
    if (a->layers > 1 && a->dst_layer_stride < a->slot_bytes) return GDR_EINVAL;
    if (a->layers > 1 && a->n_dst > 1 &&
        (__int128)a->dst_stride * (a->n_dst - 1) + a->slot_bytes > a->dst_layer_stride &&
        (__int128)a->dst_layer_stride * (a->layers - 1) + a->slot_bytes > a->dst_stride)
        return GDR_EINVAL;
    if (a->n == 0 || a->layers == 0 || a->slot_bytes == 0) return GDR_OK;
    if (!a->dst || !a->src || !a->states || !a->source) return GDR_EINVAL;
    if (!aligned16(a->states) || !aligned16(a->source)) return GDR_EINVAL;
    const CopyParams p = {(char *)a->states, (const char *)a->source, a->dst, a->src,
                          a->n_dst > 1 ? a->dst_stride : 0, a->n_src > 1 ? a->src_stride : 0, a->dst_layer_stride,
                          a->src_layer_stride, a->slot_bytes, a->layers, (int)a->n, (int)a->n_dst, (int)a->n_src};
    return done(launch_copy(p, stream));
}

}  // extern "C"
