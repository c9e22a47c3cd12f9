// Host side of the group norm (include/gdr.h): argument validation and launches.
#include "gdr_norm.hpp"

using namespace gdr;

namespace {

bool aligned16(const void *p) { return ((uintptr_t)p & 15) == 0; }

// Workgroups of a launch, four waves each: forwards eight to a compute unit; backwards four, each of which
// also writes its sums of weight and bias gradients (32768 x 8192 in bf16: 526 us with four or eight, and
// 16 or 30 for their sums)
constexpr int64_t FWD_WORKGROUPS = 256 * 8, BWD_WORKGROUPS = 256 * 4;

template <typename Args> int check(const Args *a) {
    if (!a || a->M < 0 || a->C < 1 || a->groups < 1 || a->C % a->groups != 0) return GDR_EINVAL;
    for (const int32_t t : {a->x_dtype, a->gate_dtype, a->out_dtype})
        if (t != GDR_BF16 && t != GDR_F32) return GDR_ENOTSUP;
    if (a->activation < GDR_ACT_NONE || a->activation > GDR_ACT_SIGMOID) return GDR_ENOTSUP;
    if (a->C / a->groups > NORM_WIDTH_MAX) return GDR_ENOTSUP;
    const int64_t limit = (int64_t)1 << 31;
    if (a->M >= limit || a->C >= limit / 64 || a->x_row < 0 || a->gate_row < 0) return GDR_EINVAL;
    return GDR_OK;
}

// elements of 4 bytes where the type is float
bool elements(const void *p, int32_t t) { return ((uintptr_t)p & (t == GDR_F32 ? 3 : 1)) == 0; }

Dt type_of(int32_t t) { return t == GDR_BF16 ? Dt::BF16 : Dt::F32; }

template <typename Args> NormParams params(const Args *a, NormVariant v) {
    NormParams p = {};
    p.x = a->x, p.gate = a->gate, p.weight = a->weight, p.bias = a->bias;
    p.M = a->M, p.x_row = a->x_row, p.gate_row = a->gate_row;
    p.groups = (int)a->groups, p.D = (int)(a->C / a->groups), p.lanes = v.lanes;
    p.act = a->activation, p.center = a->center != 0, p.eps = a->eps;
    return p;
}

NormGrid bwd_grid(const gdr_norm_bwd_args *a, NormVariant v) { return norm_grid(a->M, a->groups, v.lanes, BWD_WORKGROUPS); }

}  // namespace

extern "C" {

int gdr_group_norm(const gdr_norm_fwd_args *a, hipStream_t stream) {
    const int rc = check(a);
    if (rc) return rc;
    if (a->M == 0) return GDR_OK;
    if (!a->x || !a->out || !elements(a->x, a->x_dtype) || !elements(a->gate, a->gate_dtype) || !elements(a->out, a->out_dtype) ||
        !elements(a->weight, GDR_F32) || !elements(a->bias, GDR_F32))
        return GDR_EINVAL;
    const bool aligned = aligned16(a->x) && aligned16(a->gate) && aligned16(a->out) && aligned16(a->weight) && aligned16(a->bias) &&
                         a->x_row % 8 == 0 && (!a->gate || a->gate_row % 8 == 0) && a->C % 8 == 0;
    const NormVariant v = norm_variant(a->C / a->groups, aligned);
    NormParams p = params(a, v);
    p.out = a->out;
    stage_events() = {nullptr, nullptr, false};
    const hipError_t e = launch_norm(type_of(a->x_dtype), type_of(a->gate_dtype), type_of(a->out_dtype), v,
                                     norm_grid(a->M, a->groups, v.lanes, FWD_WORKGROUPS), p, stream);
    stage_events() = {nullptr, nullptr, false};
    return e == hipSuccess ? GDR_OK : GDR_ELAUNCH;
}

// parts: an upper bound for either variant
static int64_t bwd_parts(const gdr_norm_bwd_args *a) {
    int64_t most = 0;
    for (const bool aligned : {false, true}) {
        const NormGrid g = bwd_grid(a, norm_variant(a->C / a->groups, aligned));
        most = most > (int64_t)g.y ? most : (int64_t)g.y;
    }
    return most;
}

int gdr_group_norm_bwd_workspace(const gdr_norm_bwd_args *a, size_t *bytes) {
    if (!bytes) return GDR_EINVAL;
    const int rc = check(a);
    if (rc) return rc;
    *bytes = sizeof(float) * 2 * (size_t)(bwd_parts(a) * a->C);
    return GDR_OK;
}

int gdr_group_norm_bwd(const gdr_norm_bwd_args *a, hipStream_t stream) {
    const int rc = check(a);
    if (rc) return rc;
    if (!elements(a->dweight, GDR_F32) || !elements(a->dbias, GDR_F32)) return GDR_EINVAL;
    if (a->M > 0 && (!a->x || !a->dout || !a->dx || (a->gate && !a->dgate) || !elements(a->x, a->x_dtype) ||
                     !elements(a->gate, a->gate_dtype) || !elements(a->dout, a->out_dtype) || !elements(a->weight, GDR_F32) ||
                     !elements(a->bias, GDR_F32) || !elements(a->dx, a->x_dtype) || !elements(a->dgate, a->gate_dtype)))
        return GDR_EINVAL;
    const bool aligned = aligned16(a->x) && aligned16(a->gate) && aligned16(a->dout) && aligned16(a->weight) && aligned16(a->bias) &&
                         aligned16(a->dx) && aligned16(a->dgate) && a->x_row % 8 == 0 && (!a->gate || a->gate_row % 8 == 0) &&
                         a->C % 8 == 0;
    const NormVariant v = norm_variant(a->C / a->groups, aligned);
    const NormGrid g = bwd_grid(a, v);
    const int64_t parts = a->M > 0 ? (int64_t)g.y : 0;
    const bool sums = (a->dweight || a->dbias) && parts > 0;
    if (sums && (!a->workspace || !aligned16(a->workspace) || a->workspace_bytes < sizeof(float) * 2 * (size_t)(bwd_parts(a) * a->C)))
        return GDR_EWORKSPACE;
    NormParams p = params(a, v);
    p.dout = a->dout, p.dx = a->dx, p.dgate = a->dgate;
    float *ws = static_cast<float *>(a->workspace);
    if (a->dweight && sums) p.part_w = ws;
    if (a->dbias && sums) p.part_b = ws + parts * a->C;
    stage_events() = {nullptr, nullptr, false};
    hipError_t e = hipSuccess;
    if (a->M > 0) e = launch_norm_bwd(type_of(a->x_dtype), type_of(a->gate_dtype), type_of(a->out_dtype), v, g, p, stream);
    if (e == hipSuccess && (a->dweight || a->dbias))
        e = launch_norm_sum(p.part_w, p.part_b, a->dweight, a->dbias, parts, a->C, stream);
    stage_events() = {nullptr, nullptr, false};
    return e == hipSuccess ? GDR_OK : GDR_ELAUNCH;
}

}  // extern "C"
