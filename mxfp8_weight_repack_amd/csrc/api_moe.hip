// api_moe.hip -- entry points of the expert layer's operators.  Arguments are checked
// here, before anything is launched; the launchers live beside their kernels.
#include <hip/hip_runtime_api.h>

#include <algorithm>

#include "api_checks.h"
#include "moe.h"

using namespace sshdp;

namespace {

bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// tokens x top_k slots and the experts they may name.
int check_slots(int64_t tokens, int32_t top_k, int32_t experts) {
  if (tokens < 0 || top_k < 1 || experts < 1) return SSHDP_ERR_ARG;
  if (experts > kMoeMaxExperts || top_k > kMoeMaxTopK || tokens > kMoeMaxSlots / top_k) return SSHDP_ERR_SCHEMA;
  return SSHDP_OK;
}

bool any(const sshdp_mx_out &o) { return o.codes || o.scales || o.codes_t || o.scales_t; }
bool half_pair(const sshdp_mx_out &o) { return !o.codes != !o.scales || !o.codes_t != !o.scales_t; }

// What sshdp_moe_gather_mxfp8 checks of its sizes and outputs; its inputs' pointers come after.
int check_gather(const sshdp_moe_gather &a) {
  if (!dtype_ok(a.dtype) || a.rows < 0 || a.cols < 0) return SSHDP_ERR_ARG;
  const int st = check_slots(a.tokens, a.top_k, a.experts);
  if (st != SSHDP_OK) return st;
  if (a.cols % 32 || a.cols > kMaxEdge || a.rows > kMaxEdge || a.ld_x < a.cols || a.ld_x > kMaxEdge ||
      a.ld_x * dtype_size(a.dtype) % 16 || (a.out.codes_t && a.rows % 32))
    return SSHDP_ERR_SCHEMA;
  return half_pair(a.out) ? SSHDP_ERR_ARG : SSHDP_OK;
}

int check_gather_pointers(const sshdp_moe_gather &a) {
  if ((a.tokens && !a.x) || !a.source || !a.offsets) return SSHDP_ERR_ARG;
  if (!aligned16(a.x) || !aligned16(a.y) || !aligned16(a.out.codes) || !aligned16(a.out.codes_t) ||
      !aligned4(a.weights) || !aligned4(a.source) || !aligned4(a.offsets))
    return SSHDP_ERR_ALIGN;
  return check_device(a.x, a.weights, a.source, a.offsets, a.y, a.out.codes, a.out.scales, a.out.codes_t, a.out.scales_t);
}

}  // namespace

extern "C" {

int sshdp_moe_rows(int64_t tokens, int32_t top_k, int32_t experts, int32_t align, int64_t *rows) {
  if (!rows || align < 1 || (align & (align - 1))) return SSHDP_ERR_ARG;
  const int st = check_slots(tokens, top_k, experts);
  if (st != SSHDP_OK) return st;
  if (align > 256) return SSHDP_ERR_SCHEMA;
  const int64_t slots = tokens * top_k, most = slots + std::min<int64_t>(slots, experts) * (align - 1);
  *rows = align < 32 ? most : (most + 127) / 128 * 128;
  return SSHDP_OK;
}

int sshdp_moe_sort_workspace(int64_t tokens, int32_t top_k, int32_t experts, int64_t *bytes) {
  if (!bytes) return SSHDP_ERR_ARG;
  const int st = check_slots(tokens, top_k, experts);
  if (st != SSHDP_OK) return st;
  *bytes = moe_sort_counts(tokens * top_k, experts) * (int64_t)sizeof(int32_t);
  return SSHDP_OK;
}

int sshdp_moe_sort(const void *ids, int32_t ids_dtype, int64_t tokens, int32_t top_k, int32_t experts, int32_t align,
                   int32_t *offsets, int32_t *place, int32_t *source, int64_t rows, void *ws, size_t ws_bytes,
                   void *stream) {
  int64_t least = 0, need = 0;
  int st = sshdp_moe_rows(tokens, top_k, experts, align, &least);
  if (st == SSHDP_OK) st = sshdp_moe_sort_workspace(tokens, top_k, experts, &need);
  if (st != SSHDP_OK) return st;
  if (ids_dtype != SSHDP_INDEX_I32 && ids_dtype != SSHDP_INDEX_I64) return SSHDP_ERR_ARG;
  if (rows < least || rows > kMaxEdge) return SSHDP_ERR_SCHEMA;
  if (!offsets || (tokens && (!ids || !place)) || (rows && !source)) return SSHDP_ERR_ARG;
  const bool i64 = ids_dtype == SSHDP_INDEX_I64;
  if (reinterpret_cast<uintptr_t>(ids) % (i64 ? 8 : 4) || !aligned4(offsets) || !aligned4(place) || !aligned4(source))
    return SSHDP_ERR_ALIGN;
  st = check_ws(ws, ws_bytes, need);
  if (st == SSHDP_OK) st = check_device(ids, offsets, place, source);
  if (st != SSHDP_OK) return st;
  const MoeSort a{ids, tokens * top_k, rows, experts, align, offsets, place, source, i64};
  return hip_status(launch_moe_sort(a, static_cast<int32_t *>(ws), static_cast<hipStream_t>(stream)));
}

int sshdp_moe_gather_mxfp8(const sshdp_moe_gather *a, void *stream) {
  if (!a) return SSHDP_ERR_ARG;
  int st = check_gather(*a);
  if (st != SSHDP_OK) return st;
  if (a->rows == 0 || a->cols == 0) return SSHDP_OK;
  if (!a->y && !any(a->out)) return SSHDP_ERR_ARG;
  st = check_gather_pointers(*a);
  if (st != SSHDP_OK) return st;
  return hip_status(launch_moe_gather(*a, static_cast<hipStream_t>(stream)));
}

int sshdp_moe_combine(const sshdp_moe_combine_args *a, void *stream) {
  if (!a || !dtype_ok(a->dtype) || a->rows < 0 || a->cols < 0) return SSHDP_ERR_ARG;
  int st = check_slots(a->tokens, a->top_k, 1);
  if (st != SSHDP_OK) return st;
  if (a->cols % 32 || a->cols > kMaxEdge || a->rows > kMaxEdge) return SSHDP_ERR_SCHEMA;
  if (a->tokens == 0 || a->cols == 0) return SSHDP_OK;
  if ((a->rows && !a->y) || !a->place || !a->out) return SSHDP_ERR_ARG;
  if (!aligned16(a->y) || !aligned16(a->residual) || !aligned16(a->out) || !aligned4(a->place) || !aligned4(a->weights))
    return SSHDP_ERR_ALIGN;
  st = check_device(a->y, a->place, a->weights, a->residual, a->out);
  if (st != SSHDP_OK) return st;
  return hip_status(launch_moe_combine(*a, static_cast<hipStream_t>(stream)));
}

int sshdp_moe_combine_backward(const sshdp_moe_combine_grad *a, void *stream) {
  if (!a) return SSHDP_ERR_ARG;
  const sshdp_moe_gather g{a->dout, a->weights, a->source, a->offsets, a->dy, a->out, a->tokens, a->rows, a->cols,
                           a->ld_dout, a->top_k, a->experts, a->dtype, 0};
  int st = check_gather(g);
  if (st != SSHDP_OK) return st;
  if (a->cols == 0 && !a->dweights) return SSHDP_OK;
  const bool rows = a->dy || any(a->out), dots = a->dweights != nullptr;
  if (!rows && !dots) return a->rows == 0 || a->tokens == 0 ? SSHDP_OK : SSHDP_ERR_ARG;
  const bool run_rows = rows && a->rows && a->cols, run_dots = dots && a->tokens;
  if (run_rows) {
    st = check_gather_pointers(g);
    if (st != SSHDP_OK) return st;
  }
  if (run_dots) {
    if (!a->place || (a->cols && !a->dout) || (a->cols && a->rows && !a->y)) return SSHDP_ERR_ARG;
    if (!aligned16(a->dout) || !aligned16(a->y) || !aligned4(a->place) || !aligned4(a->dweights)) return SSHDP_ERR_ALIGN;
    st = check_device(a->dout, a->y, a->place, a->dweights);
    if (st != SSHDP_OK) return st;
  }
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (run_rows) {
    st = hip_status(launch_moe_gather(g, s));
    if (st != SSHDP_OK) return st;
  }
  return run_dots ? hip_status(launch_moe_dweights(*a, s)) : SSHDP_OK;
}

}  // extern "C"
