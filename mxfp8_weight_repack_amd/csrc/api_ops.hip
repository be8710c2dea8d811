// api_ops.hip -- entry points of the operators around the update: gradient norm
// and clip, MXFP8 quantisation, the residual RMS norm and its gradient, and the
// MXFP8 products.  Arguments are checked here, before anything is launched; the
// launchers live beside their kernels.
#include <hip/hip_runtime_api.h>

#include "internal.h"

using namespace sshdp;

namespace {

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int hip_status(hipError_t e) { return e == hipSuccess ? SSHDP_OK : SSHDP_ERR_HIP; }

int check_plan(const sshdp_plan *p) {
  if (!p) return SSHDP_ERR_ARG;
  if (p->host_only) return SSHDP_ERR_STATE;
  int cur = -1;
  if (hipGetDevice(&cur) != hipSuccess) return SSHDP_ERR_HIP;
  if (cur != p->device) return SSHDP_ERR_ARG;
  return SSHDP_OK;
}

// Whether a kernel on the current device may be given `p`: the device's own
// memory, or host memory the runtime allocated (NULL passes: optional tensors).
bool on_device(int cur, const void *p) {
  if (!p) return true;
  hipPointerAttribute_t a{};
  if (hipPointerGetAttributes(&a, p) != hipSuccess) {
    (void)hipGetLastError();                         // an address the runtime does not know
    return false;
  }
  if (a.type == hipMemoryTypeDevice) return a.device == cur;
  return a.type == hipMemoryTypeHost || a.type == hipMemoryTypeManaged;
}

template <class... P>
int check_device(const P *...p) {
  int cur = -1;
  if (hipGetDevice(&cur) != hipSuccess) return SSHDP_ERR_HIP;
  return (on_device(cur, p) && ...) ? SSHDP_OK : SSHDP_ERR_ARG;
}

bool dtype_ok(int32_t d) { return d == SSHDP_DTYPE_FP32 || d == SSHDP_DTYPE_BF16; }

int64_t dtype_size(int32_t d) { return d == SSHDP_DTYPE_BF16 ? 2 : 4; }

// A norm's weight, or its gradient: at any element of its array.
bool aligned_element(const void *p, int32_t d) { return reinterpret_cast<uintptr_t>(p) % dtype_size(d) == 0; }

int check_ws(const void *ws, size_t bytes, int64_t need) {
  if (need == 0) return SSHDP_OK;
  if (!ws || bytes < (size_t)need) return SSHDP_ERR_WORKSPACE;
  if (!aligned16(ws)) return SSHDP_ERR_ALIGN;
  return check_device(ws);
}

constexpr int64_t kMaxEdge = 1ll << 30;              // rows and columns of a matrix
constexpr int64_t kMaxNormCols = 32768;              // a row is held in one workgroup's registers

int64_t grad_ws(const sshdp_plan *p) { return grad_partials((int64_t)p->gchunks.size()) * (int64_t)sizeof(double); }

// Region rules of a matrix (those of a plan's MXFP8 region at offset 0), codes and
// scales present unless it is empty.
int check_matrix(const sshdp_mx_matrix *m) {
  if (!m || m->rows < 0 || m->cols < 0) return SSHDP_ERR_ARG;
  if (m->layout != SSHDP_SCALE_ROWMAJOR && m->layout != SSHDP_SCALE_TILE32X4 && m->layout != SSHDP_SCALE_BLOCK32X32)
    return SSHDP_ERR_ARG;
  if (m->rows && m->cols && (!m->codes || !m->scales)) return SSHDP_ERR_ARG;
  if (m->cols % 32 || m->rows > kMaxEdge || m->cols > kMaxEdge) return SSHDP_ERR_SCHEMA;
  if (m->layout == SSHDP_SCALE_TILE32X4 && (m->rows % 32 || m->cols % 128)) return SSHDP_ERR_SCHEMA;
  if (m->layout == SSHDP_SCALE_BLOCK32X32 && m->rows % 32) return SSHDP_ERR_SCHEMA;
  return SSHDP_OK;
}

// The MXFP8 region that a node at element o is, or whole rows of; NULL if none.  A region's
// codes and scales then hold the node's from o on in every layout, as its first row and row
// count are multiples of 32 where 32 rows share a word run or a scale.
const QRegion *region_of(const sshdp_plan &p, const sshdp_node &nd, int64_t o) {
  if (nd.rows > 1 && nd.row_stride != nd.cols) return nullptr;
  for (const QRegion &q : p.qregions) {
    const int64_t at = o - q.abs;
    if (nd.cols != q.cols || at < 0 || at % q.cols || at / q.cols + nd.rows > q.rows) continue;
    if (p.opts.scale_layout != SSHDP_SCALE_ROWMAJOR && (at / q.cols % 32 || nd.rows % 32)) return nullptr;
    return &q;
  }
  return nullptr;
}

int check_gemm(const sshdp_mx_matrix *a, const sshdp_mx_matrix *b, int32_t op) {
  int st = check_matrix(a);
  if (st != SSHDP_OK) return st;
  st = check_matrix(b);
  if (st != SSHDP_OK) return st;
  if (op != SSHDP_GEMM_NT && op != SSHDP_GEMM_NN) return SSHDP_ERR_ARG;
  if (a->cols != (op == SSHDP_GEMM_NN ? b->rows : b->cols) || a->cols > (1 << 22)) return SSHDP_ERR_SCHEMA;
  if (op == SSHDP_GEMM_NN && (b->layout != SSHDP_SCALE_BLOCK32X32 || b->cols > (1 << 23))) return SSHDP_ERR_SCHEMA;
  return SSHDP_OK;
}

}  // namespace

extern "C" {

int sshdp_grad_workspace(const sshdp_plan *p, int64_t *bytes) {
  if (!p || !bytes) return SSHDP_ERR_ARG;
  *bytes = grad_ws(p);
  return SSHDP_OK;
}

int sshdp_grad_sumsq(const sshdp_plan *p, const float *grad, double *sumsq, void *ws, size_t ws_bytes, void *stream) {
  int st = check_plan(p);
  if (st != SSHDP_OK) return st;
  if (!grad || !sumsq) return SSHDP_ERR_ARG;
  if (!aligned16(grad) || !aligned16(sumsq)) return SSHDP_ERR_ALIGN;
  st = check_ws(ws, ws_bytes, grad_ws(p));
  if (st == SSHDP_OK) st = check_device(grad, sumsq);
  if (st != SSHDP_OK) return st;
  hipStream_t s = static_cast<hipStream_t>(stream);
  st = hip_status(launch_grad_partials(*p, grad, static_cast<double *>(ws), s));
  if (st != SSHDP_OK) return st;
  return hip_status(launch_grad_total(*p, static_cast<double *>(ws), sumsq, s));
}

int sshdp_grad_clip(const sshdp_plan *p, const float *grad, float *out, const double *sumsq, float max_norm,
                    float *stats, void *stream) {
  int st = check_plan(p);
  if (st != SSHDP_OK) return st;
  if (!grad || !out || !sumsq || !stats || !(max_norm > 0.f)) return SSHDP_ERR_ARG;
  if (!aligned16(grad) || !aligned16(out) || !aligned16(sumsq) || !aligned16(stats)) return SSHDP_ERR_ALIGN;
  st = check_device(grad, out, sumsq, stats);
  if (st != SSHDP_OK) return st;
  return hip_status(launch_grad_scale(*p, grad, out, sumsq, 1, max_norm, stats, static_cast<hipStream_t>(stream)));
}

int sshdp_grad_clip_norm(const sshdp_plan *p, const float *grad, float *out, float max_norm, float *stats, void *ws,
                         size_t ws_bytes, void *stream) {
  int st = check_plan(p);
  if (st != SSHDP_OK) return st;
  if (!grad || !out || !stats || !(max_norm > 0.f)) return SSHDP_ERR_ARG;
  if (!aligned16(grad) || !aligned16(out) || !aligned16(stats)) return SSHDP_ERR_ALIGN;
  const int64_t need = grad_ws(p);
  st = check_ws(ws, ws_bytes, need);
  if (st == SSHDP_OK) st = check_device(grad, out, stats);
  if (st != SSHDP_OK) return st;
  hipStream_t s = static_cast<hipStream_t>(stream);
  double *parts = static_cast<double *>(ws);
  st = hip_status(launch_grad_partials(*p, grad, parts, s));
  if (st != SSHDP_OK) return st;
  return hip_status(launch_grad_scale(*p, grad, out, parts, need / (int64_t)sizeof(double), max_norm, stats, s));
}

int sshdp_quant_mxfp8(const void *src, int32_t dtype, int64_t rows, int64_t cols, int64_t ld, uint8_t *codes,
                      uint8_t *scales, uint8_t *codes_t, uint8_t *scales_t, void *stream) {
  if (!dtype_ok(dtype) || rows < 0 || cols < 0) return SSHDP_ERR_ARG;
  if (cols % 32 || ld < cols || ld * dtype_size(dtype) % 16 || rows > kMaxEdge || ld > kMaxEdge)
    return SSHDP_ERR_SCHEMA;
  if (rows == 0 || cols == 0) return SSHDP_OK;
  if (!src || !codes != !scales || !codes_t != !scales_t || (!codes && !codes_t)) return SSHDP_ERR_ARG;
  if (!aligned16(src) || !aligned16(codes) || !aligned16(codes_t)) return SSHDP_ERR_ALIGN;
  const int st = check_device(src, codes, scales, codes_t, scales_t);
  if (st != SSHDP_OK) return st;
  const bool bf16 = dtype == SSHDP_DTYPE_BF16;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (!codes_t) return hip_status(launch_quant_rows(src, bf16, rows, cols, ld, codes, scales, s));
  return hip_status(launch_quant_tiles(src, bf16, rows, cols, ld, codes, scales, codes_t, scales_t, s));
}

int sshdp_rmsnorm_mxfp8(const sshdp_rmsnorm *a, void *stream) {
  if (!a || !dtype_ok(a->dtype) || !dtype_ok(a->weight_dtype) || a->rows < 0 || a->cols < 0 || !(a->eps >= 0.f))
    return SSHDP_ERR_ARG;
  const int64_t es = dtype_size(a->dtype);
  if (a->cols % 32 || a->cols > kMaxNormCols || a->rows > kMaxEdge || a->ld_x < a->cols || a->ld_x > kMaxEdge ||
      a->ld_x * es % 16)
    return SSHDP_ERR_SCHEMA;
  if (a->residual && (a->ld_residual < a->cols || a->ld_residual > kMaxEdge || a->ld_residual * es % 16))
    return SSHDP_ERR_SCHEMA;
  if (a->rows == 0 || a->cols == 0) return SSHDP_OK;
  if (!a->x || !a->weight || !a->codes != !a->scales || (a->h && !a->residual)) return SSHDP_ERR_ARG;
  if (!a->h && !a->y && !a->codes && !a->rstd) return SSHDP_ERR_ARG;
  // h is dense: written over rows with gaps it would run into rows not read yet
  if (a->h && a->rows > 1 &&
      ((a->h == a->x && a->ld_x != a->cols) || (a->h == a->residual && a->ld_residual != a->cols)))
    return SSHDP_ERR_SCHEMA;
  if (!aligned16(a->x) || !aligned16(a->residual) || !aligned_element(a->weight, a->weight_dtype) || !aligned16(a->h) ||
      !aligned16(a->y) || !aligned16(a->codes) || !aligned16(a->rstd))
    return SSHDP_ERR_ALIGN;
  const int st = check_device(a->x, a->residual, a->weight, a->h, a->y, a->codes, a->scales, a->rstd);
  if (st != SSHDP_OK) return st;
  return hip_status(launch_rmsnorm(*a, static_cast<hipStream_t>(stream)));
}

int sshdp_rmsnorm_backward_workspace(int64_t rows, int64_t cols, int64_t *bytes) {
  if (!bytes || rows < 0 || cols < 0) return SSHDP_ERR_ARG;
  if (cols % 32 || cols > kMaxNormCols || rows > kMaxEdge) return SSHDP_ERR_SCHEMA;
  *bytes = rows == 0 ? 0 : rmsnorm_partials(rows, cols) * cols * (int64_t)sizeof(float);
  return SSHDP_OK;
}

int sshdp_rmsnorm_backward(const sshdp_rmsnorm_grad *a, void *ws, size_t ws_bytes, void *stream) {
  if (!a || !dtype_ok(a->dtype) || !dtype_ok(a->weight_dtype)) return SSHDP_ERR_ARG;
  int64_t need = 0;
  int st = sshdp_rmsnorm_backward_workspace(a->rows, a->cols, &need);
  if (st != SSHDP_OK) return st;
  if (a->cols == 0 || (a->rows == 0 && !a->first)) return SSHDP_OK;
  if (!a->dweight) return SSHDP_ERR_ARG;
  if (a->rows && (!a->dy || !a->h || !a->weight || !a->rstd || !a->dx)) return SSHDP_ERR_ARG;
  if (!aligned16(a->dy) || !aligned16(a->h) || !aligned16(a->dh) || !aligned_element(a->weight, a->weight_dtype) ||
      !aligned16(a->rstd) || !aligned16(a->dx) || !aligned_element(a->dweight, SSHDP_DTYPE_FP32))
    return SSHDP_ERR_ALIGN;
  st = check_ws(ws, ws_bytes, need);
  if (st == SSHDP_OK) st = check_device(a->dy, a->h, a->dh, a->weight, a->rstd, a->dx, a->dweight);
  if (st != SSHDP_OK) return st;
  return hip_status(launch_rmsnorm_backward(*a, static_cast<float *>(ws), static_cast<hipStream_t>(stream)));
}

int sshdp_plan_mx_matrix(const sshdp_plan *p, int32_t node, const uint8_t *codes, const uint8_t *scales,
                         sshdp_mx_matrix *out) {
  if (!p || !out || !codes || !scales || node < 0 || node >= (int32_t)p->nodes.size()) return SSHDP_ERR_ARG;
  const sshdp_node &nd = p->nodes[node];
  const int64_t o = p->node_abs[node];
  const QRegion *region = region_of(*p, nd, o);
  if (!region) return SSHDP_ERR_SCHEMA;
  out->codes = codes + o;
  out->scales = scales + o / (p->opts.scale_layout == SSHDP_SCALE_BLOCK32X32 ? 1024 : 32);
  out->rows = nd.rows;
  out->cols = nd.cols;
  out->layout = p->opts.scale_layout;
  out->pad_ = 0;
  return SSHDP_OK;
}

int sshdp_gemm_mxfp8_workspace(const sshdp_mx_matrix *a, const sshdp_mx_matrix *b, int32_t op, int64_t *bytes) {
  if (!bytes) return SSHDP_ERR_ARG;
  const int st = check_gemm(a, b, op);
  if (st != SSHDP_OK) return st;
  const bool nn = op == SSHDP_GEMM_NN;
  *bytes = gemm_mx_workspace(a->rows, nn ? b->cols : b->rows, a->cols, nn);
  return SSHDP_OK;
}

int sshdp_gemm_mxfp8(const sshdp_mx_matrix *a, const sshdp_mx_matrix *b, int32_t op, const float *addend, void *out,
                     int32_t out_dtype, int64_t ld_out, void *ws, size_t ws_bytes, void *stream) {
  int64_t need = 0;
  int st = sshdp_gemm_mxfp8_workspace(a, b, op, &need);
  if (st != SSHDP_OK) return st;
  if (!dtype_ok(out_dtype) || (addend && out_dtype != SSHDP_DTYPE_FP32)) return SSHDP_ERR_ARG;
  GemmMx g{};
  g.nn = op == SSHDP_GEMM_NN;
  g.m = a->rows;
  g.n = g.nn ? b->cols : b->rows;
  g.k = a->cols;
  if (ld_out < g.n || ld_out > kMaxEdge) return SSHDP_ERR_SCHEMA;
  if (g.m == 0 || g.n == 0) return SSHDP_OK;
  if (!out) return SSHDP_ERR_ARG;
  if (!aligned16(a->codes) || !aligned16(b->codes) || !aligned16(addend) || !aligned16(out)) return SSHDP_ERR_ALIGN;
  st = check_ws(ws, ws_bytes, need);
  if (st == SSHDP_OK) st = check_device(a->codes, a->scales, b->codes, b->scales, addend, out);
  if (st != SSHDP_OK) return st;
  g.a = a->codes;
  g.as = a->scales;
  g.la = a->layout;
  g.b = b->codes;
  g.bs = b->scales;
  g.lb = b->layout;
  g.addend = addend;
  g.out = out;
  g.ld = ld_out;
  g.bf16 = out_dtype == SSHDP_DTYPE_BF16;
  return hip_status(launch_gemm_mx(g, ws, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
