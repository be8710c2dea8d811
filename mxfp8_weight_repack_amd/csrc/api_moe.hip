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

constexpr int64_t kMaxTiles = 1 << 22;

// B of a product of experts' rows: groups equal parts, each a matrix by the layout's rules.
int check_bank(const sshdp_mx_matrix &b, int32_t groups) {
  if (b.rows % groups) return SSHDP_ERR_SCHEMA;
  return b.layout != SSHDP_SCALE_ROWMAJOR && b.rows / groups % 32 ? SSHDP_ERR_SCHEMA : SSHDP_OK;
}

int check_groups(const int32_t *offsets, int32_t groups) {
  if (groups < 1 || (!offsets && groups != 1)) return SSHDP_ERR_ARG;
  return groups > kMoeMaxExperts ? SSHDP_ERR_SCHEMA : SSHDP_OK;
}

// The operands' part of a grouped product, checked.
int make_grouped(const sshdp_mx_matrix *a, const sshdp_mx_matrix *b, GroupForm form, const int32_t *offsets,
                 int32_t groups, GemmGrouped &g) {
  int st = check_matrix(a);
  if (st == SSHDP_OK) st = check_matrix(b);
  if (st == SSHDP_OK) st = check_groups(offsets, groups);
  if (st != SSHDP_OK) return st;
  if (a->layout != SSHDP_SCALE_ROWMAJOR) return SSHDP_ERR_SCHEMA;
  g.form = form;
  g.offsets = offsets;
  g.groups = groups;
  g.p.a = a->codes;
  g.p.as = a->scales;
  g.p.b = b->codes;
  g.p.bs = b->scales;
  g.p.la = a->layout;
  g.p.lb = b->layout;
  g.p.nn = form == kRowsNN;
  g.p.m = a->rows;
  g.p.k = a->cols;
  if (form == kColumns) {
    if (b->layout != SSHDP_SCALE_ROWMAJOR || a->cols != b->cols || a->cols % 128) return SSHDP_ERR_SCHEMA;
    g.p.n = b->rows;
  } else {
    st = check_bank(*b, groups);
    if (st != SSHDP_OK) return st;
    const int64_t rows = b->rows / groups;
    if (a->cols != (g.p.nn ? rows : b->cols) || a->cols == 0) return SSHDP_ERR_SCHEMA;
    if (g.p.nn && (b->layout != SSHDP_SCALE_BLOCK32X32 || b->cols > (1 << 23) || (rows >> 5) * (b->cols >> 5) < 4))
      return SSHDP_ERR_SCHEMA;
    g.p.n = g.p.nn ? b->cols : rows;
  }
  if (a->cols > (1 << 22)) return SSHDP_ERR_SCHEMA;
  return grouped_tiles(form, groups, g.p.m, g.p.n, 128) > kMaxTiles ? SSHDP_ERR_SCHEMA : SSHDP_OK;
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

int sshdp_gemm_mxfp8_grouped(const sshdp_mx_matrix *a, const sshdp_mx_matrix *b, int32_t op, const int32_t *offsets,
                             int32_t groups, const void *addend, void *out, int32_t out_dtype, int64_t ld_out,
                             void *stream) {
  if (op != SSHDP_GEMM_NT && op != SSHDP_GEMM_NN && op != SSHDP_GEMM_TN) return SSHDP_ERR_ARG;
  const bool tn = op == SSHDP_GEMM_TN;
  if (!dtype_ok(out_dtype) || (tn && out_dtype != SSHDP_DTYPE_FP32)) return SSHDP_ERR_ARG;
  GemmGrouped g{};
  int st = make_grouped(a, b, tn ? kColumns : op == SSHDP_GEMM_NN ? kRowsNN : kRowsNT, offsets, groups, g);
  if (st != SSHDP_OK) return st;
  if (ld_out < g.p.n || ld_out > kMaxEdge) return SSHDP_ERR_SCHEMA;
  if (g.p.m == 0 || g.p.n == 0) return SSHDP_OK;
  if (!out) return SSHDP_ERR_ARG;
  if (!aligned16(a->codes) || !aligned16(b->codes) || !aligned16(addend) || !aligned16(out) || !aligned4(offsets))
    return SSHDP_ERR_ALIGN;
  st = check_device(a->codes, a->scales, b->codes, b->scales, offsets, addend, out);
  if (st != SSHDP_OK) return st;
  g.bf16 = out_dtype == SSHDP_DTYPE_BF16;
  g.p.out = out;
  g.p.ld = ld_out;
  g.p.bf16 = g.bf16;
  if (g.bf16) g.addend16 = static_cast<const uint16_t *>(addend);
  else g.p.addend = static_cast<const float *>(addend);
  return hip_status(launch_gemm_grouped(g, static_cast<hipStream_t>(stream)));
}

int sshdp_gemm_mxfp8_swiglu(const sshdp_mx_matrix *a, const sshdp_mx_matrix *gate_w, const sshdp_mx_matrix *up_w,
                            const int32_t *offsets, int32_t groups, uint8_t *codes, uint8_t *scales, void *gate,
                            void *up, void *stream) {
  GemmGrouped g{};
  int st = check_matrix(up_w);
  if (st == SSHDP_OK) st = make_grouped(a, gate_w, kRowsGated, offsets, groups, g);
  if (st != SSHDP_OK) return st;
  if (up_w->rows != gate_w->rows || up_w->cols != gate_w->cols || up_w->layout != gate_w->layout || g.p.n % 32)
    return SSHDP_ERR_SCHEMA;
  if (g.p.m == 0 || g.p.n == 0) return SSHDP_OK;
  if (!codes != !scales || !gate != !up || (!codes && !gate)) return SSHDP_ERR_ARG;
  if (!aligned16(a->codes) || !aligned16(gate_w->codes) || !aligned16(up_w->codes) || !aligned16(codes) ||
      !aligned16(gate) || !aligned16(up) || !aligned4(offsets))
    return SSHDP_ERR_ALIGN;
  st = check_device(a->codes, a->scales, gate_w->codes, gate_w->scales, up_w->codes, up_w->scales, offsets, codes,
                    scales, gate, up);
  if (st != SSHDP_OK) return st;
  g.bf16 = g.p.bf16 = true;
  g.p.ld = g.p.n;
  g.b2 = up_w->codes;
  g.b2s = up_w->scales;
  g.codes = codes;
  g.scales = scales;
  g.gate = static_cast<uint16_t *>(gate);
  g.up = static_cast<uint16_t *>(up);
  return hip_status(launch_gemm_grouped(g, static_cast<hipStream_t>(stream)));
}

int sshdp_swiglu_backward_mxfp8(const sshdp_swiglu_grad *a, void *stream) {
  if (!a || a->rows < 0 || a->cols < 0) return SSHDP_ERR_ARG;
  const sshdp_mx_out *outs[] = {&a->dgate, &a->dup, &a->h};
  bool columns = false;
  for (const sshdp_mx_out *o : outs) {
    if (half_pair(*o)) return SSHDP_ERR_ARG;
    columns = columns || o->codes_t;
  }
  if (a->offsets) {
    const int st = check_groups(a->offsets, a->groups);
    if (st != SSHDP_OK) return st;
  }
  if (a->cols % 32 || a->cols > kMaxEdge || a->rows > kMaxEdge || (columns && a->rows % 32)) return SSHDP_ERR_SCHEMA;
  if (a->rows == 0 || a->cols == 0) return SSHDP_OK;
  const bool grads = any(a->dgate) || any(a->dup);
  if (!a->gate || !a->up || (grads && !a->dh) || (!grads && !any(a->h))) return SSHDP_ERR_ARG;
  if (!aligned16(a->dh) || !aligned16(a->gate) || !aligned16(a->up) || !aligned4(a->offsets)) return SSHDP_ERR_ALIGN;
  for (const sshdp_mx_out *o : outs)
    if (!aligned16(o->codes) || !aligned16(o->codes_t)) return SSHDP_ERR_ALIGN;
  int st = check_device(a->dh, a->gate, a->up, a->offsets);
  for (const sshdp_mx_out *o : outs)
    if (st == SSHDP_OK) st = check_device(o->codes, o->scales, o->codes_t, o->scales_t);
  if (st != SSHDP_OK) return st;
  return hip_status(launch_swiglu_grad(*a, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
