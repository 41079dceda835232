// C ABI of the steps around the grouped GEMMs: argument validation and
// dispatch to their kernels. The contract is documented in include/moe/dg_moe.h.

#include "../../include/moe/dg_moe.h"

#include <hip/hip_runtime.h>

#include "dg_moe_internal.h"

namespace {

using namespace dg::moe;

constexpr long long kMaxBytes = 1LL << 40;
constexpr long long kMaxSlots = 1LL << 22;  // this and the next two keep workgroups * threads of every grid below 2^32
constexpr int kMaxGluRows = 1 << 22;
constexpr long long kMaxRows = 1LL << 30;
constexpr int kMaxNormTokens = 1 << 21;
constexpr int kMaxDim = 1 << 20;

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4b(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

dg_status status_of(hipError_t e) { return e == hipSuccess ? DG_OK : DG_ERR_LAUNCH; }
// The kernels are built for gfx950 only: no usable device, no launch.
dg_status device_check() { return dg_get_num_cus() > 0 ? DG_OK : DG_ERR_DEVICE; }
hipStream_t as_stream(void* s) { return reinterpret_cast<hipStream_t>(s); }

// Sizes of a row layout with `m` rows (a group, where masked).
dg_status layout_checks(int layout, int m, int num_groups) {
  if (layout < DG_MOE_CONTIGUOUS || layout > DG_MOE_NOPAD || num_groups <= 0 || m < 0) return DG_ERR_SHAPE;
  if (layout == DG_MOE_MASKED && m == 0) return DG_ERR_SHAPE;
  if (layout == DG_MOE_CONTIGUOUS && m % SEGMENT != 0) return DG_ERR_SHAPE;
  if (num_groups > (layout == DG_MOE_NOPAD ? MAX_NOPAD : MAX_GROUPS)) return DG_ERR_UNSUPPORTED;
  // Row numbers are ints, and a kernel's loop over rows steps past the last one.
  if ((long long)m * (layout == DG_MOE_MASKED ? num_groups : 1) >= kMaxRows) return DG_ERR_UNSUPPORTED;
  return DG_OK;
}

dg_status plan_sizes(const dg_moe_plan* p) {
  if (!p) return DG_ERR_NULL;
  if (dg_status s = layout_checks(p->layout, p->rows, p->num_groups)) return s;
  if (p->max_tokens < 0 || p->top_k <= 0 || p->hidden <= 0 || p->hidden % QBLOCK != 0) return DG_ERR_SHAPE;
  if (p->top_k > MAX_TOP_K || p->hidden > kMaxDim || (long long)p->max_tokens * p->top_k > kMaxSlots)
    return DG_ERR_UNSUPPORTED;
  const long long rows = (long long)p->rows * (p->layout == DG_MOE_MASKED ? p->num_groups : 1);
  if (rows * p->hidden * 2 >= kMaxBytes || (long long)p->max_tokens * p->hidden * 2 >= kMaxBytes)
    return DG_ERR_UNSUPPORTED;
  return DG_OK;
}

long long plan_workspace(const dg_moe_plan* p) {
  return 16 + sort_workspace(p->max_tokens * p->top_k, p->num_groups);
}

dg_status plan_checks(const dg_moe_plan* p, int tokens, RouteArgs& a) {
  if (dg_status s = plan_sizes(p)) return s;
  if (tokens < 0 || tokens > p->max_tokens) return DG_ERR_SHAPE;
  if ((!p->row_of && p->max_tokens > 0) || !p->group_rows || !p->workspace) return DG_ERR_NULL;
  if (p->layout == DG_MOE_CONTIGUOUS && p->rows > 0 && !p->grouped_layout) return DG_ERR_NULL;
  if (!aligned4b(p->row_of) || !aligned4b(p->group_rows) || !aligned4b(p->grouped_layout) || !aligned16(p->workspace))
    return DG_ERR_ALIGN;
  if (p->workspace_bytes < plan_workspace(p)) return DG_ERR_SHAPE;
  a = RouteArgs{};
  a.layout = p->layout;
  a.tokens = tokens;
  a.top_k = p->top_k;
  a.num_groups = p->num_groups;
  a.rows = p->rows;
  a.hidden = p->hidden;
  a.row_of = p->row_of;
  a.group_rows = p->group_rows;
  a.grouped_layout = p->layout == DG_MOE_CONTIGUOUS ? p->grouped_layout : nullptr;
  a.workspace = p->workspace;
  return DG_OK;
}

// Buffers of `tokens` or of the permuted rows may be null only if empty.
bool missing(const void* p, long long count) { return !p && count > 0; }

dg_status glu_checks(const int32_t* rows, int layout, int m, int num_groups, int inner) {
  if (layout == DG_MOE_DENSE) {
    if (m < 0) return DG_ERR_SHAPE;
  } else {
    if (dg_status s = layout_checks(layout, m, layout == DG_MOE_CONTIGUOUS ? 1 : num_groups)) return s;
    if (!rows && m > 0) return DG_ERR_NULL;
    if (!aligned4b(rows)) return DG_ERR_ALIGN;
  }
  if (inner <= 0 || inner % QBLOCK != 0) return DG_ERR_SHAPE;
  if (inner > kMaxDim || m > kMaxGluRows) return DG_ERR_UNSUPPORTED;
  const long long all = (long long)m * (layout == DG_MOE_MASKED ? num_groups : 1);
  if (all * inner * 4 >= kMaxBytes) return DG_ERR_UNSUPPORTED;
  return DG_OK;
}

dg_status norm_sizes(int tokens, int hidden, int gate_kind) {
  if (tokens < 0 || hidden <= 0 || hidden % 8 != 0) return DG_ERR_SHAPE;
  if (gate_kind < DG_MOE_GATE_NONE || gate_kind > DG_MOE_GATE_FULL) return DG_ERR_SHAPE;
  if (hidden > MAX_NORM_HIDDEN || tokens > kMaxNormTokens) return DG_ERR_UNSUPPORTED;
  return DG_OK;
}

bool gate_aligned(const void* gate, int kind) { return kind == DG_MOE_GATE_TOKEN ? aligned4b(gate) : aligned16(gate); }

}  // namespace

extern "C" {

long long dg_moe_workspace_bytes(const dg_moe_plan* plan) {
  return plan_sizes(plan) == DG_OK ? plan_workspace(plan) : -1;
}

dg_status dg_moe_sort(const dg_moe_plan* plan, const int32_t* topk_ids, int tokens, void* stream) {
  RouteArgs a;
  if (dg_status s = plan_checks(plan, tokens, a)) return s;
  if (missing(topk_ids, tokens)) return DG_ERR_NULL;
  if (!aligned4b(topk_ids)) return DG_ERR_ALIGN;
  a.ids = topk_ids;
  if (dg_status s = device_check()) return s;
  return status_of(launch_sort(a, as_stream(stream)));
}

dg_status dg_moe_dispatch(const dg_moe_plan* plan, const int32_t* topk_ids, const void* x, void* xp, int tokens,
                          void* stream) {
  RouteArgs a;
  if (dg_status s = plan_checks(plan, tokens, a)) return s;
  if (missing(x, tokens) || missing(xp, (long long)tokens * a.rows)) return DG_ERR_NULL;
  if (!aligned16(x) || !aligned16(xp) || !aligned4b(topk_ids)) return DG_ERR_ALIGN;
  a.ids = topk_ids;
  if (tokens == 0 && !topk_ids) return DG_OK;
  if (dg_status s = device_check()) return s;
  return status_of(launch_dispatch(a, x, xp, as_stream(stream)));
}

dg_status dg_moe_dispatch_fp8(const dg_moe_plan* plan, const int32_t* topk_ids, const void* x, void* q, float* sfa,
                              int tokens, int ue8m0, void* stream) {
  RouteArgs a;
  if (dg_status s = plan_checks(plan, tokens, a)) return s;
  if (missing(x, tokens) || missing(q, (long long)tokens * a.rows) || missing(sfa, (long long)tokens * a.rows))
    return DG_ERR_NULL;
  if (!aligned16(x) || !aligned16(q) || !aligned16(sfa) || !aligned4b(topk_ids)) return DG_ERR_ALIGN;
  a.ids = topk_ids;
  if (tokens == 0 && !topk_ids) return DG_OK;
  if (dg_status s = device_check()) return s;
  return status_of(launch_dispatch_fp8(a, x, q, sfa, ue8m0 != 0, as_stream(stream)));
}

dg_status dg_moe_combine(const dg_moe_plan* plan, const void* yp, const float* weights, void* y, int tokens,
                         void* stream) {
  RouteArgs a;
  if (dg_status s = plan_checks(plan, tokens, a)) return s;
  if (missing(yp, (long long)tokens * a.rows) || missing(y, tokens)) return DG_ERR_NULL;
  if (!aligned16(yp) || !aligned16(y) || !aligned4b(weights)) return DG_ERR_ALIGN;
  if (tokens == 0) return DG_OK;
  if (dg_status s = device_check()) return s;
  return status_of(launch_combine(a, yp, weights, y, as_stream(stream)));
}

dg_status dg_moe_combine_bwd(const dg_moe_plan* plan, const void* dy, const void* yp, const float* weights, void* dyp,
                             float* dweights, int tokens, void* stream) {
  RouteArgs a;
  if (dg_status s = plan_checks(plan, tokens, a)) return s;
  const long long any = (long long)tokens * a.rows;
  if (missing(dy, tokens) || missing(weights, tokens) || missing(dyp, any)) return DG_ERR_NULL;
  if (dweights && missing(yp, any)) return DG_ERR_NULL;
  if (!aligned16(dy) || !aligned16(yp) || !aligned16(dyp) || !aligned4b(weights) || !aligned4b(dweights))
    return DG_ERR_ALIGN;
  if (tokens == 0) return DG_OK;
  if (dg_status s = device_check()) return s;
  return status_of(launch_combine_bwd(a, dy, yp, weights, dyp, dweights, as_stream(stream)));
}

dg_status dg_moe_swiglu_fp8(const void* gu, void* q, float* sfa, const int32_t* rows, int layout, int m,
                            int num_groups, int inner, int ue8m0, void* stream) {
  if (dg_status s = glu_checks(rows, layout, m, num_groups, inner)) return s;
  if (missing(gu, m) || missing(q, m) || missing(sfa, m)) return DG_ERR_NULL;
  if (!aligned16(gu) || !aligned16(q) || !aligned16(sfa)) return DG_ERR_ALIGN;
  if (m == 0) return DG_OK;
  GluArgs a{};
  a.gu = static_cast<const uint16_t*>(gu);
  a.q = static_cast<uint8_t*>(q);
  a.sfa = sfa;
  a.rows = rows;
  a.layout = layout;
  a.m = m;
  a.num_groups = num_groups;
  a.inner = inner;
  if (dg_status s = device_check()) return s;
  return status_of(launch_swiglu_fp8(a, ue8m0 != 0, as_stream(stream)));
}

dg_status dg_moe_swiglu_bwd(const void* da, const void* gu, void* dgu, const int32_t* rows, int layout, int m,
                            int num_groups, int inner, void* stream) {
  if (dg_status s = glu_checks(rows, layout, m, num_groups, inner)) return s;
  if (missing(da, m) || missing(gu, m) || missing(dgu, m)) return DG_ERR_NULL;
  if (!aligned16(da) || !aligned16(gu) || !aligned16(dgu)) return DG_ERR_ALIGN;
  if (m == 0) return DG_OK;
  GluArgs a{};
  a.gu = static_cast<const uint16_t*>(gu);
  a.da = static_cast<const uint16_t*>(da);
  a.dgu = static_cast<uint16_t*>(dgu);
  a.rows = rows;
  a.layout = layout;
  a.m = m;
  a.num_groups = num_groups;
  a.inner = inner;
  if (dg_status s = device_check()) return s;
  return status_of(launch_swiglu_bwd(a, as_stream(stream)));
}

dg_status dg_moe_block_norm(const dg_moe_norm* args, void* stream) {
  if (!args) return DG_ERR_NULL;
  const dg_moe_norm& a = *args;
  if (dg_status s = norm_sizes(a.tokens, a.hidden, a.gate_kind)) return s;
  if (!(a.eps >= 0.0f)) return DG_ERR_SHAPE;
  if (a.tokens == 0) return DG_OK;
  if (!a.x || (!a.y && !a.n)) return DG_ERR_NULL;
  // What a missing part would use has to be missing too, and the rest there.
  if ((a.gate_kind == DG_MOE_GATE_NONE) != (a.gate == nullptr)) return DG_ERR_NULL;
  if (a.y && !a.h) return DG_ERR_NULL;
  if (!a.y && (a.h || a.gate || a.post_weight || a.residual_scale != 1.0f)) return DG_ERR_NULL;
  if (!a.post_weight && a.rstd_post) return DG_ERR_NULL;
  if (a.n ? !a.pre_weight : (a.pre_weight || a.rstd_pre)) return DG_ERR_NULL;
  for (const void* p : {a.x, a.y, (const void*)a.post_weight, (const void*)a.pre_weight, (const void*)a.h,
                        (const void*)a.n})
    if (!aligned16(p)) return DG_ERR_ALIGN;
  if (!gate_aligned(a.gate, a.gate_kind) || !aligned4b(a.rstd_post) || !aligned4b(a.rstd_pre)) return DG_ERR_ALIGN;
  const int cus = dg_get_num_cus();
  if (cus <= 0) return DG_ERR_DEVICE;
  return status_of(launch_block_norm(a, cus, as_stream(stream)));
}

long long dg_moe_block_norm_workspace_bytes(int tokens, int hidden) {
  if (norm_sizes(tokens, hidden, DG_MOE_GATE_NONE) != DG_OK) return -1;
  return 16 + (long long)norm_bwd_grid(tokens) * 2 * hidden * 4;
}

dg_status dg_moe_block_norm_bwd(const dg_moe_norm_bwd* args, void* stream) {
  if (!args) return DG_ERR_NULL;
  const dg_moe_norm_bwd& a = *args;
  if (dg_status s = norm_sizes(a.tokens, a.hidden, a.gate_kind)) return s;
  if (!a.workspace) return DG_ERR_NULL;
  if (a.tokens > 0) {
    if ((!a.dh && !a.dn) || !a.dx) return DG_ERR_NULL;
    if ((a.gate_kind == DG_MOE_GATE_NONE) != (a.gate == nullptr)) return DG_ERR_NULL;
    if (a.dn ? (!a.h || !a.pre_weight || !a.rstd_pre) : (a.pre_weight || a.rstd_pre || a.dpre_weight))
      return DG_ERR_NULL;
    if (a.y ? !a.dy : (a.dy || a.gate || a.post_weight || a.residual_scale != 1.0f)) return DG_ERR_NULL;
    if (a.post_weight ? !a.rstd_post : (a.rstd_post || a.dpost_weight)) return DG_ERR_NULL;
    if (!a.gate && a.dgate) return DG_ERR_NULL;
  }
  for (const void* p : {a.dh, a.dn, a.h, a.y, (const void*)a.post_weight, (const void*)a.pre_weight,
                        (const void*)a.dx, (const void*)a.dy, (const void*)a.workspace})
    if (!aligned16(p)) return DG_ERR_ALIGN;
  if (!gate_aligned(a.gate, a.gate_kind) || !gate_aligned(a.dgate, a.gate_kind)) return DG_ERR_ALIGN;
  if (!aligned4b(a.rstd_post) || !aligned4b(a.rstd_pre) || !aligned4b(a.dpost_weight) || !aligned4b(a.dpre_weight))
    return DG_ERR_ALIGN;
  if (a.workspace_bytes < dg_moe_block_norm_workspace_bytes(a.tokens, a.hidden)) return DG_ERR_SHAPE;
  const int cus = dg_get_num_cus();
  if (cus <= 0) return DG_ERR_DEVICE;
  return status_of(launch_block_norm_bwd(a, cus, as_stream(stream)));
}

}  // extern "C"
