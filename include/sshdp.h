/*
 * sshdp.h -- C ABI of libsshdp.so: one GPU's share of the SS-HSDP update phase
 * on MI355X (gfx950).
 *
 * Sources, cited by title and section:
 *   [SS-HSDP]  "SS-HSDP: Efficient and Flexible Sharded Data Parallelism via
 *              Runtime-Update Decoupling" (arXiv:2611.16467v1)
 *   [OCP-MX]   OCP Microscaling Formats (MX) v1.0, the MXFP format cited there
 *
 * What the library computes.  [SS-HSDP §2.1]: an optimizer update F maps
 * (main weight, main gradient, optimizer state) to new main weight and state,
 * and weight preparation G casts or quantises the main weight into the
 * low-precision runtime weight and its scales.  [SS-HSDP §3.1, EG1]: for Muon,
 * F = [f0, f1, f2] per update unit (one attention head, one matrix): f0 updates
 * the momentum and writes a BF16 intermediate u, f1 runs Newton-Schulz on u and
 * produces an FP32 direction v, f2 updates the main weight from v; G produces
 * FP8 (E4M3) weights with UE8M0 scales, and the weight transform Tw packs the
 * head weights into the runtime weight (a view, no copy [SS-HSDP §3.2, §4.2])
 * and relays the scales out for the GEMM kernel.  [SS-HSDP §5.2]: AdamW updates
 * the parameters Muon does not.
 *
 * Data model.  Every field (main weight, gradient, momentum, AdamW second
 * moment, FP8 codes) is ONE flat root allocation indexed by the same element
 * offsets; views are described by a data tree [SS-HSDP §3.2 "Data Tree"]: a
 * child is a view at an element offset inside its parent, only the root owns
 * storage.  Codes mirror the fp32 root byte-for-element, so a head's codes are a
 * sub-range of its packed projection's codes.  Scales are one E8M0 byte per
 * 1x32 block (row-major or the 32x128 tile layout) or per 32x32 block (see
 * SSHDP_SCALE_*).
 *
 * Conventions.  All functions return an int status: SSHDP_OK (0) or a negative
 * SSHDP_ERR_* code; sshdp_status_string() names it.  Device pointers are
 * caller-owned, must stay valid until the enqueued work has run, and must be
 * 16-byte aligned unless a function says less.  `stream` is a hipStream_t passed as void* (NULL = the
 * default stream); every launching call is asynchronous on it, performs no
 * allocation and no synchronisation.  Newton-Schulz groups of one call may run
 * on up to three plan-owned side streams (default priority) that are forked
 * from and joined back into `stream` with events, so the call behaves as one
 * ordered unit of work on `stream` (and can be captured into a HIP graph).
 * Calls with one plan use its side streams: issue them from one host thread,
 * in order (their work is then ordered as issued).  Calls sharing a workspace
 * are serialised by the caller's stream order.  The library keeps no state
 * between calls: the step counter is an argument.
 */
#ifndef SSHDP_H
#define SSHDP_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define SSHDP_ABI_VERSION 6

/* Status codes.  The planning errors are the rejections of [SS-HSDP Appendix A,
 * Table 4]: incompatible metadata, invalid geometry, storage overlap. */
enum {
  SSHDP_OK = 0,
  SSHDP_ERR_ARG = -1,       /* null pointer, empty table, step < 1, bad option value   */
  SSHDP_ERR_TREE = -2,      /* a parent index is not an earlier node                   */
  SSHDP_ERR_BOUNDS = -3,    /* a view leaves its parent or the root                    */
  SSHDP_ERR_OVERLAP = -4,   /* two units, or two quantised regions, share an element   */
  SSHDP_ERR_SCHEMA = -5,    /* geometry/metadata the kernels cannot take (see below)   */
  SSHDP_ERR_ALIGN = -6,     /* a device pointer is not 16-byte aligned                 */
  SSHDP_ERR_WORKSPACE = -7, /* workspace missing or smaller than sshdp_plan_info says  */
  SSHDP_ERR_HIP = -8,       /* a HIP runtime call or kernel launch failed              */
  SSHDP_ERR_STATE = -9,     /* the plan was made host-only and cannot launch           */
  SSHDP_ERR_SCRATCH = -10   /* the plan needs more workspace than the built-in scratch  */
};

enum { SSHDP_OPT_NONE = 0, SSHDP_OPT_MUON = 1, SSHDP_OPT_ADAMW = 2 };

/* Scale layouts.  For a quantised region at absolute element offset o with N
 * rows and K columns (KB = K/32 blocks per row), the scale of block (n, kb):
 *   ROWMAJOR : o/32 + n*KB + kb             (= index of its first element / 32)
 *   TILE32X4 : o/32 + ((n/32)*(KB/4) + kb/4)*128 + (n%32)*4 + kb%4
 * TILE32X4 stores each 32-row x 128-column tile's scales as one 128-byte run,
 * one 4-byte word per row holding 4 consecutive K-blocks: the operand a 32-row
 * scaled-MFMA tile reads in one coalesced load.  It is this library's own
 * layout (the [SS-HSDP] kernels' layout belongs to other hardware).  Both
 * layouts keep a head's scales a sub-range of its projection's when the head's
 * row count is a multiple of 32.
 *
 * BLOCK32X32 is the other block shape [SS-HSDP §3.1 EG1] (and [veScale §6])
 * describe: one scale per 32-row x 32-column block, the least-e rule over the
 * block's 1024 elements, codes as above; block (bn, bk) of a region at o with
 * K columns has its scale at  o/1024 + bn*(K/32) + bk.  The blocks of X^T are
 * the transposes of X's, so the same codes serve the transposed operand.  The
 * scale array then holds (root_numel + 1023)/1024 bytes, and AdamW is never
 * fused with G (the AdamW units run first, then G). */
enum { SSHDP_SCALE_ROWMAJOR = 0, SSHDP_SCALE_TILE32X4 = 1, SSHDP_SCALE_BLOCK32X32 = 2 };

/* Plan flags.  The Newton-Schulz tile policy is a tuning knob (results stay
 * within the Newton-Schulz tolerance either way, not bit-identical): by default
 * a group's products run in 256 x 256 tiles over their largest 256-aligned
 * leading block when the group is large enough to fill the GPU with them, and
 * in 128 x 128 tiles elsewhere.  Setting both tile flags is an argument error.
 * Gram products that run in 128-tiles read X^T (so only X^T is stored) unless
 * SSHDP_PLAN_NS_GRAM_NT is set or X^T of the unit exceeds 2^31 bytes.  Groups
 * other than the largest run on side streams while the largest group's
 * launches fill fewer than two rounds of the GPU's workgroup slots in some
 * stage; otherwise only the groups with r_pad == 128 do (on one side stream)
 * and the rest share the caller's stream.  SSHDP_PLAN_NS_ONE_STREAM keeps
 * every group on the caller's stream. */
enum {
  SSHDP_PLAN_HOST_ONLY = 1,       /* plan and validate on the host; no device tables (cannot launch) */
  SSHDP_PLAN_NS_TILES_SMALL = 2,  /* every Newton-Schulz product in 128 x 128 tiles                  */
  SSHDP_PLAN_NS_TILES_LARGE = 4,  /* 256 x 256 tiles over every 256-aligned leading block            */
  SSHDP_PLAN_NS_GRAM_NT = 8,      /* every Gram reads X row-major (X and X^T stored); for comparison */
  SSHDP_PLAN_NS_ONE_STREAM = 16   /* every Newton-Schulz group on the caller's stream, none on side streams */
};

/* One data-tree node [SS-HSDP §3.2]: a 2-D view (rows x cols, cols contiguous,
 * rows `row_stride` elements apart) at `offset` elements from its parent's first
 * element.  A 1-D tensor is rows = 1.  `is_unit` marks an update parameter (a
 * leaf of the optimisation [SS-HSDP §3.1]) with `optimizer` SSHDP_OPT_MUON or
 * SSHDP_OPT_ADAMW; `quantize` marks a region (a runtime weight, or a unit)
 * that G turns into its runtime form [SS-HSDP §2.1: G casts or quantises the
 * main weight]: SSHDP_G_MXFP8 requantises it to MXFP8 (codes + scales),
 * SSHDP_G_BF16 casts it to bfloat16 (w_bf16).  Rules (else the error named):
 *   parent is -1 or an earlier node index                          (TREE)
 *   rows, cols >= 1, offset >= 0, row_stride >= cols if rows > 1   (SCHEMA)
 *   the view lies inside its parent's extent and the root           (BOUNDS)
 *   a Muon unit is 2-D (rows, cols >= 2) and its first element, row_stride
 *     and cols are multiples of 4 (16-byte vectors); rows, cols <= 4194176
 *     (a 256-row bf16 panel of that length spans < 2^31 bytes)     (SCHEMA)
 *   quantize is SSHDP_G_NONE, SSHDP_G_MXFP8 or SSHDP_G_BF16          (SCHEMA)
 *   an MXFP8 region is contiguous (row_stride == cols), with cols and its
 *     first element multiples of 32; for TILE32X4 also rows % 32 == 0 and
 *     cols % 128 == 0; for BLOCK32X32 also rows % 32 == 0 and the
 *     first element a multiple of 1024                              (SCHEMA)
 *   a BF16 region is contiguous, with cols and its first element
 *     multiples of 8 (16-byte stores)                               (SCHEMA)
 *   units are pairwise disjoint; G regions (both kinds) too        (OVERLAP)
 * Checks run node by node in index order; overlap is checked last. */
typedef struct {
  int32_t parent;
  int32_t is_unit;
  int64_t offset;
  int64_t rows;
  int64_t cols;
  int64_t row_stride;
  int32_t optimizer;
  int32_t quantize;
} sshdp_node;

enum { SSHDP_G_NONE = 0, SSHDP_G_MXFP8 = 1, SSHDP_G_BF16 = 2 };

/* Plan options.  Defaults (sshdp_default_opts): 5 Newton-Schulz steps with
 * (a, b, c) = (3.4445, -4.7750, 2.0315) on the Frobenius-normalised u, ns_eps =
 * 1e-7 added to the norm, heavy-ball momentum (nesterov = 0), update scale mode
 * 0 (scale 1; mode 1: sqrt(max(1, rows/cols)); mode 2: 0.2*sqrt(max(rows,
 * cols))), ROWMAJOR scales, flags 0. */
typedef struct {
  int32_t ns_steps;
  float ns_a, ns_b, ns_c;
  float ns_eps;
  int32_t scale_layout;
  int32_t nesterov;
  int32_t muon_scale_mode;
  uint32_t flags;
} sshdp_plan_opts;

/* Muon: m <- momentum*m + g; u = bf16(m) (nesterov: bf16(g + momentum*m));
 * v = NS(u); w <- w - lr*weight_decay*w - lr*scale*v. */
typedef struct { float lr, momentum, weight_decay; } sshdp_muon_hp;

/* AdamW: w <- w - lr*wd*w; m <- b1 m + (1-b1) g; v <- b2 v + (1-b2) g^2;
 * w <- w - lr * (m/(1-b1^t)) / (sqrt(v/(1-b2^t)) + eps). */
typedef struct { float lr, beta1, beta2, eps, weight_decay; } sshdp_adamw_hp;

/* Caller-owned device roots, all indexed by the same element offsets.
 * w_main, grad, mom (Muon momentum and AdamW first moment): fp32, root_numel
 * elements.  adam_v: fp32 root or NULL when the plan has no AdamW units.
 * codes: uint8 root of root_numel bytes (E4M3FN).  scales: uint8, at least
 * sshdp_plan_stats.scale_bytes bytes (E8M0).  w_bf16: bfloat16 root of
 * root_numel elements, or NULL when the plan has no BF16 regions.  Only unit
 * elements of w_main, mom, adam_v, MXFP8-region bytes of codes/scales and
 * BF16-region elements of w_bf16 are written. */
typedef struct {
  float *w_main;
  const float *grad;
  float *mom;
  float *adam_v;
  uint8_t *codes;
  uint8_t *scales;
  uint16_t *w_bf16;
} sshdp_buffers;

typedef struct sshdp_plan sshdp_plan;   /* opaque; owns host tables and one device table block */

/* Figures a caller needs to size buffers, and the algorithmic work per step. */
typedef struct {
  int64_t root_numel;
  int64_t scale_bytes;        /* bytes of the scale root: ceil(root_numel / 32)            */
  int64_t workspace_bytes;    /* device workspace sshdp_update_muon/_step need (256-aligned) */
  int32_t n_nodes, n_units, n_muon_units, n_adamw_units, n_quant_regions, n_groups;
  int64_t muon_elems, adamw_elems, quant_elems;
  int64_t fused_quant_elems;  /* MXFP8 elements G handles inside the AdamW pass           */
  double ns_flops;            /* steps*(4 r^2 c + 2 r^3) summed over Muon units: the dense count */
  double ns_tile_flops;       /* MFMA flops the tile schedule executes per step (symmetric Gram and
                                 poly computed as tm <= tn tiles; padding to the tile included; units
                                 whose momentum is all zero skip theirs at run time)             */
  int64_t cast_elems;         /* elements of BF16 regions                                  */
  int32_t n_cast_regions;
  int32_t pad_;
} sshdp_plan_stats;

/* One Newton-Schulz batch: the Muon units sharing an oriented shape r x c
 * (r = min(rows, cols)), run as one batched GEMM per stage [SS-HSDP §4.1]. */
typedef struct {
  int32_t r, c;               /* oriented shape                                            */
  int32_t r_pad, c_pad;       /* padded to a multiple of 128                               */
  int32_t n_units;
  int32_t tile;               /* largest macro-tile edge of the update product (128 or 256) */
  int32_t tile_gram;          /* largest macro-tile edge of the Gram and polynomial products */
  int32_t gram256;            /* Gram/poly rows and columns [0, gram256) run in 256-tiles,  */
                              /* the rest in 128-tiles (0: all 128)                          */
  int32_t upd256_rows;        /* update rows [0, upd256_rows) x columns [0, upd256_cols)    */
  int32_t upd256_cols;        /* run in 256-tiles, the rest in 128-tiles                     */
  int32_t gram_kmajor;        /* 1: the Gram reads X^T (K-major) and X itself is not stored  */
  int32_t split_b;            /* 1 (groups with r_pad == 128): the polynomial B goes to memory  */
                              /* as a bf16 pair, its rounding and the remainder, and the update */
                              /* contracts over both (twice the update's K)                     */
  int32_t lane;               /* stream the group runs on: 0 = the caller's, 1.. = side streams */
} sshdp_group_info;

/* Fill *opts with the defaults above. */
int sshdp_default_opts(sshdp_plan_opts *opts);

/* Resolve the data tree and build a plan [SS-HSDP §3.2 "Data Tree"; §3.3
 * groups; Appendix A Table 4 rejections].  Host-synchronous; unless
 * SSHDP_PLAN_HOST_ONLY, allocates and uploads one block of device descriptor
 * tables on the current HIP device.  Errors leave *out_plan NULL and touch no
 * device memory.  The plan is freed by sshdp_plan_destroy, which releases its
 * device tables and side streams: call it only once the work enqueued with the
 * plan has completed. */
int sshdp_plan_views(const sshdp_node *nodes, int32_t n_nodes, int64_t root_numel,
                     const sshdp_plan_opts *opts, sshdp_plan **out_plan);

int sshdp_plan_info(const sshdp_plan *plan, sshdp_plan_stats *stats);
int sshdp_plan_group(const sshdp_plan *plan, int32_t group, sshdp_group_info *info);
/* Absolute element offset of node `node` (accumulated along its chain) and the
 * Newton-Schulz group of a Muon unit (-1 otherwise). */
int sshdp_plan_node(const sshdp_plan *plan, int32_t node, int64_t *abs_offset, int32_t *group);
void sshdp_plan_destroy(sshdp_plan *plan);

/* F for every Muon unit: f0 (momentum, bf16 u, ||u||^2), f1 (Newton-Schulz,
 * batched bf16 MFMA GEMMs per group) and f2 (main-weight update, fused into the
 * last Newton-Schulz product) [SS-HSDP §3.1 EG1, §4.1].  Reads grad, mom,
 * w_main; writes mom, w_main.  `workspace`: device memory of at least
 * stats.workspace_bytes, 256-byte aligned; its contents on entry are ignored.
 * Errors (nothing is launched): ARG (null plan/bufs/hp/grad/mom/w_main, or the
 * current device is not the plan's), STATE (host-only plan), ALIGN, WORKSPACE
 * (null or too small); HIP if a launch fails. */
int sshdp_update_muon(const sshdp_plan *plan, const sshdp_buffers *bufs, const sshdp_muon_hp *hp,
                      void *workspace, size_t workspace_bytes, void *stream);

/* F for every AdamW unit at step `step` (>= 1, caller-owned, same for all
 * units) [SS-HSDP §5.2: the parameters Muon does not take -- 1-D and
 * elementwise ones -- are updated by AdamW; Appendix B.1: AdamW is the
 * optimizer of every performance run].  The pages write no AdamW formula; the
 * form is the sshdp_adamw_hp one above (decay lr*wd on the pre-update weight,
 * bias-corrected moments, eps after the square root), elementwise in fp32.
 * Reads grad, mom, adam_v, w_main; writes mom, adam_v, w_main.
 * Errors: ARG (null pointers, step < 1, wrong device), STATE, ALIGN; HIP. */
int sshdp_update_adamw(const sshdp_plan *plan, const sshdp_buffers *bufs, const sshdp_adamw_hp *hp,
                       int64_t step, void *stream);

/* G + the scale part of Tw for every quantised region [SS-HSDP §3.1 EG1; OCP-MX]:
 * per 1x32 block along K, e = least integer with amax <= 448*2^e (clamped to
 * [-127,127]; all-zero block -> -127), scale byte e+127 at the layout's index,
 * codes = E4M3FN round-to-nearest-even of x*2^-e, written at the elements' own
 * offsets.  A block holding NaN/Inf gets scale 0xFF and codes 0x7F.  Reads
 * w_main; writes codes and scales.  A plan without MXFP8 regions returns OK at
 * once.  Errors: ARG (null pointers, wrong device), STATE, ALIGN (w_main or
 * codes); HIP. */
int sshdp_requant_mxfp8(const sshdp_plan *plan, const float *w_main, uint8_t *codes, uint8_t *scales,
                        void *stream);

/* G for every BF16 region [SS-HSDP §2.1]: w_bf16 = bfloat16(w_main), round to
 * nearest even, at the elements' own offsets (a runtime view of a BF16 weight
 * is the same sub-range of w_bf16).  Reads w_main; writes w_bf16.  A plan
 * without BF16 regions returns OK at once.  Errors: ARG, STATE, ALIGN; HIP. */
int sshdp_cast_bf16(const sshdp_plan *plan, const float *w_main, uint16_t *w_bf16, void *stream);

/* The reduce-scatter tail [SS-HSDP §4.3 "Reduce-Scatter", Figure 5(e)]: within
 * a node, the slices of one output partition arriving from several ranks are
 * summed in FP32 by a local reducer; the partial stays FP32 or, for BF16
 * gradients, is stored as BF16 with stochastic rounding; the final FP32
 * reduction accumulates straight into the persistent gradient buffer (G'z2),
 * with no result buffer and no separate addition pass.  On one GPU the slices
 * are device buffers (what peer copies deliver).
 *
 * `inputs`: host array of n_inputs (1..8) device pointers, each n elements of
 * in_dtype (SSHDP_RS_FP32 or SSHDP_RS_BF16), summed left to right, every
 * addition rounded to FP32.  n % 16 == 0 and every pointer 16-byte aligned.
 *
 * sshdp_rs_reduce writes the sum to `out` as FP32 (SSHDP_RS_OUT_FP32) or as
 * BF16 with stochastic rounding (SSHDP_RS_OUT_BF16_SR): the fp32 bit pattern
 * plus a 16-bit random, truncated to its upper half (NaN kept), i.e. away from
 * zero with probability (discarded bits)/2^16.  The randoms come from
 * Philox4x64-10 [Salmon et al., SC 2011] with key (seed, 0): element j of the
 * call is element g = g0 + j of the whole tensor (g0 % 16 == 0) and uses word
 * (g/4) % 4, bits 16*(g%4), of the block at counter (g/16 + 1, ctr, 0, 0) --
 * so a rank that restores (seed, ctr) reproduces its partials.
 *
 * sshdp_rs_accumulate: g = in_0 + in_1 + ... when `first` (the first
 * microbatch initialises the buffer), else g = (g + in_0) + in_1 + ....
 *
 * Errors: ARG (null pointer, n_inputs out of range, n < 0, bad dtype/mode),
 * SCHEMA (n or g0 not a multiple of 16), ALIGN. */
enum { SSHDP_RS_FP32 = 0, SSHDP_RS_BF16 = 1 };
enum { SSHDP_RS_OUT_FP32 = 0, SSHDP_RS_OUT_BF16_SR = 1 };
int sshdp_rs_reduce(const void *const *inputs, int32_t n_inputs, int32_t in_dtype, void *out, int32_t out_mode,
                    int64_t n, uint64_t seed, uint64_t ctr, int64_t g0, void *stream);
int sshdp_rs_accumulate(const void *const *inputs, int32_t n_inputs, int32_t in_dtype, float *g, int64_t n,
                        int32_t first, void *stream);

/* The whole update phase in order [SS-HSDP §3.4 "Update"]: Muon F, AdamW F
 * (fused with G for MXFP8 regions holding only AdamW units; the other AdamW
 * units may run on a plan-owned side stream beside the Newton-Schulz work, as
 * they share no element with a Muon unit), then G for the remaining MXFP8
 * regions and the BF16 regions.  Equivalent to
 * sshdp_update_muon; sshdp_update_adamw; sshdp_requant_mxfp8; sshdp_cast_bf16.
 * Every argument the plan's parts need is checked before anything is launched
 * (the errors of those calls); mh may be NULL for a plan without Muon units
 * and ah for one without AdamW units. */
int sshdp_update_step(const sshdp_plan *plan, const sshdp_buffers *bufs, const sshdp_muon_hp *mh,
                      const sshdp_adamw_hp *ah, int64_t step, void *workspace, size_t workspace_bytes,
                      void *stream);

/* sshdp_update_step without caller workspace, for callers that cannot
 * allocate device memory (code under HIP graph capture, tight serving loops,
 * harnesses that forbid hipMalloc).  The workspace is a device array built
 * into the library, SSHDP_NOALLOC_SCRATCH_BYTES (64 MiB) on every GPU the
 * library runs on, held until the process ends; its address is looked up on
 * the first call on each device.  The call allocates nothing (with
 * sshdp_profile_enable on, its timing events are created on first use, as in
 * every launching call).  Plans whose stats.workspace_bytes exceed the array
 * are refused (SSHDP_ERR_SCRATCH) before anything is launched.  Every call on
 * a GPU shares that GPU's array and leaves its contents behind (nothing in it
 * needs to start at zero: each step writes the whole region it reads), so
 * calls that may overlap on one GPU -- on different streams or from different
 * threads -- race; order them on one stream.  Otherwise it is exactly
 * sshdp_update_step: same arguments, results and other errors. */
#define SSHDP_NOALLOC_SCRATCH_BYTES (64u << 20)
int sshdp_update_step_noalloc(const sshdp_plan *plan, const sshdp_buffers *bufs, const sshdp_muon_hp *mh,
                              const sshdp_adamw_hp *ah, int64_t step, void *stream);

/* Operators around the update: what the gradient passes through before it, and
 * what reads the MXFP8 runtime weights it leaves behind.  They follow the
 * conventions above (asynchronous on `stream`, no allocation, no
 * synchronisation, caller-owned workspace whose contents on entry are ignored,
 * capturable).  Every tensor must be memory of the current device, else ARG;
 * outputs must not overlap inputs except where said.  Where a call has nothing
 * to do (no rows), it returns OK and its tensors may be NULL. */

/* The global gradient norm over every unit of the plan, and clipping by it
 * (the step between the reduce-scatter tail and F).  sumsq = sum of g^2 over
 * all unit elements, held in float64 from the first product on (no overflow
 * for any finite float32 gradient); norm = sqrt(sumsq); coef = max_norm / norm
 * if norm > max_norm, else 1 (an infinite norm gives coef 0, a NaN norm 1: the
 * caller sees the norm in `stats` and skips the step).  out = g * coef on unit
 * elements; `out` may be `grad` itself (then a coef of 1 writes nothing).
 * Elements outside the units are neither read nor written.
 *
 * sshdp_grad_clip_norm does all of it; `stats` receives two floats, norm and
 * coef.  A norm over several GPUs' shards takes it in two steps:
 * sshdp_grad_sumsq writes this GPU's sum to one double (16-byte aligned), the
 * caller adds the ranks' sums up, and sshdp_grad_clip clips by that total.
 * Sums are added in a fixed order: the same gradient gives the same bits.
 * `workspace`: sshdp_grad_workspace(plan) bytes, 16-byte aligned.
 * Errors: ARG (null pointer, max_norm not > 0, wrong device), STATE, ALIGN,
 * WORKSPACE; HIP. */
int sshdp_grad_workspace(const sshdp_plan *plan, int64_t *bytes);
int sshdp_grad_sumsq(const sshdp_plan *plan, const float *grad, double *sumsq, void *workspace,
                     size_t workspace_bytes, void *stream);
int sshdp_grad_clip(const sshdp_plan *plan, const float *grad, float *out, const double *sumsq, float max_norm,
                    float *stats, void *stream);
int sshdp_grad_clip_norm(const sshdp_plan *plan, const float *grad, float *out, float max_norm, float *stats,
                         void *workspace, size_t workspace_bytes, void *stream);

/* Element types of the matrices below. */
enum { SSHDP_DTYPE_FP32 = 0, SSHDP_DTYPE_BF16 = 1 };

/* G of any matrix: src (rows x cols of `dtype`, rows `ld` elements apart) to
 * MXFP8 along its rows, along its columns, or both in one pass over it:
 *   codes   rows x cols, scales rows x cols/32: blocks of 32 along a row, the
 *           rule and rounding of sshdp_requant_mxfp8, scales ROWMAJOR;
 *   codes_t cols x R, scales_t cols x R/32 with R = rows rounded up to 32: the
 *           transpose, blocks of 32 along src's columns; the last block's
 *           missing rows count as zeros and get code 0.
 * Pass NULL for a pair not wanted.  These are the operands of a linear layer's
 * products: activations and output gradients along their rows, and along the
 * tokens for the weight gradient.
 * Errors: ARG (null src, half a pair or no pair, bad dtype, rows or cols < 0),
 * SCHEMA (cols not a multiple of 32, ld < cols, ld rows not 16-byte multiples,
 * an edge over 2^30), ALIGN (src, codes, codes_t; scales: any); HIP. */
int sshdp_quant_mxfp8(const void *src, int32_t dtype, int64_t rows, int64_t cols, int64_t ld, uint8_t *codes,
                      uint8_t *scales, uint8_t *codes_t, uint8_t *scales_t, void *stream);

/* RMS norm of rows, with the residual's addition in front and G behind:
 *   h = x + residual, rounded to `dtype` (without residual: h = x);
 *   rstd = 1 / sqrt(mean(h^2) + eps) of each row;
 *   y = h * rstd * weight, rounded to float32; codes, scales = G(y) along rows.
 * The row statistics and y's products are held in float64, so y is the correct
 * float32 but for products within 2^-29 of a rounding border, and its codes
 * follow the oracle's bit for bit.  Outputs are dense (rows x cols; scales
 * ROWMAJOR rows x cols/32), each NULL if not wanted, codes and scales together:
 * `h` (only with residual; may be x or residual where that one is dense), `y` in
 * `dtype`, and `rstd`, one float per row (what the backward needs).  x and
 * residual have rows ld_x and ld_residual elements apart; `weight` has cols
 * elements of weight_dtype and may start at any of them (a norm unit's place in
 * the main-weight or bfloat16 root).
 * A NaN makes its whole row's y NaN; an infinity makes rstd 0, y NaN where it
 * stands and 0 elsewhere; G gives blocks holding NaN scale 0xFF and codes 0x7F.
 * Errors: ARG (null x or weight, no output, half a pair, h without residual,
 * bad dtype, eps < 0 or NaN, rows or cols < 0), SCHEMA (cols not a multiple of
 * 32 or over 32768, ld < cols, rows not 16-byte multiples, h in place of rows
 * with gaps), ALIGN; HIP. */
typedef struct {
  const void *x, *residual, *weight;
  void *h, *y;
  uint8_t *codes, *scales;
  float *rstd;
  int64_t rows, cols, ld_x, ld_residual;
  int32_t dtype, weight_dtype;
  float eps;
  int32_t pad_;
} sshdp_rmsnorm;
int sshdp_rmsnorm_mxfp8(const sshdp_rmsnorm *args, void *stream);

/* Its gradient (G passes gradients straight through).  With xhat = h * rstd:
 *   dx = rstd * (weight dy - xhat mean(weight dy xhat)) + dh;
 *   dweight = sum over rows of dy * xhat, added to what is there unless `first`.
 * dx is the gradient of x and of the residual alike; `dh` (optional) is the
 * gradient reaching h past the norm.  dy, h, dh, dx are dense rows x cols of
 * `dtype`; dweight is float32 (a norm unit's place in the gradient root, at any
 * element of it: 4-byte aligned).  dx may be dy or dh.  Sums are held in float32 and added in a fixed order.
 * `workspace`: sshdp_rmsnorm_backward_workspace bytes, 16-byte aligned.
 * rows == 0: dweight is set to 0 if `first`, else left.
 * Errors: ARG (null pointer but dh, bad dtype), SCHEMA (as above), ALIGN,
 * WORKSPACE; HIP. */
typedef struct {
  const void *dy, *h, *dh, *weight;
  const float *rstd;
  void *dx;
  float *dweight;
  int64_t rows, cols;
  int32_t dtype, weight_dtype, first, pad_;
} sshdp_rmsnorm_grad;
int sshdp_rmsnorm_backward_workspace(int64_t rows, int64_t cols, int64_t *bytes);
int sshdp_rmsnorm_backward(const sshdp_rmsnorm_grad *args, void *workspace, size_t workspace_bytes, void *stream);

/* A matrix in MXFP8: dense row-major codes and scales in one of the
 * SSHDP_SCALE_* layouts (the region formulas with o = 0, from `scales` on).
 * sshdp_plan_mx_matrix describes a node of a plan inside the codes and scales
 * roots, so a product reads the runtime weight where G left it: an MXFP8 region,
 * or a view of whole rows of one (an expert of a bank, a head of a packed
 * projection), whatever node carries `quantize`.  In the layouts that group 32
 * rows the view starts at a multiple of 32 of the region's rows and has a
 * multiple of 32.  Errors: ARG (null pointer, no such node), SCHEMA (any other
 * node). */
typedef struct {
  const uint8_t *codes, *scales;
  int64_t rows, cols;
  int32_t layout, pad_;
} sshdp_mx_matrix;
int sshdp_plan_mx_matrix(const sshdp_plan *plan, int32_t node, const uint8_t *codes, const uint8_t *scales,
                         sshdp_mx_matrix *out);

/* The MXFP8 product of a linear layer, on the matrix cores:
 *   SSHDP_GEMM_NT: out[m][n] = sum_k A[m][k] B[n][k]  (A M x K, B N x K): the
 *     forward product (A activations, B the weight), or the weight gradient
 *     (both operands quantised along the tokens);
 *   SSHDP_GEMM_NN: out[m][n] = sum_k A[m][k] B[k][n]  (B K x N, BLOCK32X32, whose
 *     scales serve both directions): the input gradient, from the very codes of
 *     the forward product.
 * out: M x N, rows ld_out elements apart, float32 or bfloat16 (round to nearest
 * even).  Float32 output is a float32 sum of exact products.  For bfloat16 output
 * the matrix cores multiply the codes themselves, twice as fast: each 8
 * consecutive k's products are cut off at 2^-14 of the binade of their largest
 * before they are added, so such a group is off by less than 7 * 2^-14 of its
 * largest product (about 1.4e-5 rms of a result of random operands).  That error
 * goes by the products: where they cancel it may exceed bfloat16's own 2^-8 of
 * the small result; take float32 output where that matters.  `addend`
 * (float32 output only, NULL for none) has out's shape and ld and is added to
 * the sums; it may be `out`: gradients of microbatches.
 * Any M and N, K a multiple of 32; K == 0 gives the addend, or zeros.  NaN
 * blocks (scale 0xFF) give NaN.  `workspace`: sshdp_gemm_mxfp8_workspace bytes
 * (0: none needed), 16-byte aligned.  The result does not depend on timing.
 * For float32 output element values (code times scale) must lie within bfloat16's
 * range: from 2^128 on they count as infinite, and under 2^-126 they lose bits and
 * then vanish (G gives such values for elements as small themselves, and for those
 * that round up to 2^128).  bfloat16 output takes every code under every scale.
 * Errors: ARG (null pointer, bad op, layout or dtype, addend with bfloat16,
 * negative size), SCHEMA (the operands' K differ, a layout's rules -- rows and
 * cols of the region rules above --, NN without BLOCK32X32, ld_out < N, M or N
 * over 2^30, K over 2^22, an NN row pitch over 2^23), ALIGN (codes, addend,
 * out), WORKSPACE; HIP. */
enum { SSHDP_GEMM_NT = 0, SSHDP_GEMM_NN = 1 };
int sshdp_gemm_mxfp8_workspace(const sshdp_mx_matrix *a, const sshdp_mx_matrix *b, int32_t op, int64_t *bytes);
int sshdp_gemm_mxfp8(const sshdp_mx_matrix *a, const sshdp_mx_matrix *b, int32_t op, const float *addend, void *out,
                     int32_t out_dtype, int64_t ld_out, void *workspace, size_t workspace_bytes, void *stream);

/* A mixture-of-experts layer on the expert banks: tokens are sorted by expert,
 * each expert's tokens pass through its own weights as consecutive rows, and the
 * results go back to their tokens.
 *
 * sshdp_moe_sort orders the tokens x top_k slots of `ids` (slot s = t * top_k + j:
 * token t's choice j; int32, or int64 if ids_dtype is SSHDP_INDEX_I64) by expert,
 * equal experts by slot.  An id outside [0, experts) drops its slot: a padding
 * token, or an expert of another GPU.  Each expert's rows start at a multiple of
 * `align` (a power of two up to 256):
 *   offsets  experts + 1: expert e has the rows offsets[e] .. offsets[e + 1] - 1,
 *            its slots first, then under `align` rows of padding;
 *   place    tokens x top_k: each slot's row, -1 if dropped;
 *   source   rows: each row's slot, -1 for padding and behind the last expert.
 * `rows` is the buffers' size, at least sshdp_moe_rows of the same sizes (the most
 * that any ids take; with align >= 32 a multiple of 128).  An expert may be chosen
 * twice by one token.  align 32 and over keeps the blocks of 32 rows that the
 * weight gradient's operands have inside one expert.  `workspace`:
 * sshdp_moe_sort_workspace bytes, 16-byte aligned.
 * Errors: ARG (null pointer, tokens < 0, top_k < 1, experts < 1, align no power of
 * two, bad dtype), SCHEMA (experts over 1024, top_k over 64, over 2^24 slots, align
 * over 256, rows too few or over 2^30), ALIGN (offsets, place, source; ids: its own
 * type's), WORKSPACE; HIP. */
enum { SSHDP_INDEX_I32 = 0, SSHDP_INDEX_I64 = 1 };
int sshdp_moe_rows(int64_t tokens, int32_t top_k, int32_t experts, int32_t align, int64_t *rows);
int sshdp_moe_sort_workspace(int64_t tokens, int32_t top_k, int32_t experts, int64_t *bytes);
int sshdp_moe_sort(const void *ids, int32_t ids_dtype, int64_t tokens, int32_t top_k, int32_t experts, int32_t align,
                   int32_t *offsets, int32_t *place, int32_t *source, int64_t rows, void *workspace,
                   size_t workspace_bytes, void *stream);

/* An MXFP8 output: codes and scales along rows, codes_t and scales_t along columns
 * (the transpose), as sshdp_quant_mxfp8 lays them out; NULL: not wanted. */
typedef struct {
  uint8_t *codes, *scales, *codes_t, *scales_t;
} sshdp_mx_out;

/* Tokens to the experts' rows: row p of the result is
 *   v[p] = weights[s] * x[s / top_k],  s = source[p]   (weights NULL: 1),
 * and zeros where source has -1 (or no slot of these tokens).  `y` receives v in
 * `dtype`, `out` G(v) of v rounded to float32: along the rows, along the columns
 * (pitch `rows`, a multiple of 32; its blocks are of 32 sorted rows), or both.
 * Rows from offsets[experts] on are left as they were (columns: blocks that start
 * there).  x has rows ld_x elements apart.  The gradient of x is sshdp_moe_combine
 * of the rows' gradients, with the same weights.
 * Errors: ARG (null x, source or offsets, no output, half a pair, bad dtype, a
 * negative size, top_k or experts < 1), SCHEMA (cols not a multiple of 32, rows not
 * one with codes_t, ld_x < cols or its rows not 16-byte multiples, an edge over
 * 2^30, experts over 1024, top_k over 64, over 2^24 slots), ALIGN (all but the
 * scales; weights, source and offsets 4); HIP. */
typedef struct {
  const void *x;
  const float *weights;
  const int32_t *source, *offsets;
  void *y;
  sshdp_mx_out out;
  int64_t tokens, rows, cols, ld_x;
  int32_t top_k, experts, dtype, pad_;
} sshdp_moe_gather;
int sshdp_moe_gather_mxfp8(const sshdp_moe_gather *args, void *stream);

/* The experts' rows back to their tokens:
 *   out[t] = residual[t] + sum over j of weights[t][j] * y[place[t][j]],
 * added up in float32 in the order of j, the residual last, rounded to `dtype`
 * once; dropped slots (a place outside [0, rows)) add nothing.  weights NULL: 1;
 * residual NULL: 0.  y is rows x cols, out and residual tokens x cols, all dense;
 * out may be residual.
 * Errors: ARG (null y, place or out, bad dtype, a negative size, top_k < 1), SCHEMA
 * (cols not a multiple of 32, an edge over 2^30, top_k over 64, over 2^24 slots),
 * ALIGN (as above); HIP. */
typedef struct {
  const void *y;
  const int32_t *place;
  const float *weights;
  const void *residual;
  void *out;
  int64_t tokens, rows, cols;
  int32_t top_k, dtype;
} sshdp_moe_combine_args;
int sshdp_moe_combine(const sshdp_moe_combine_args *args, void *stream);

/* Its gradient.  dy[p] = weights[s] * dout[s / top_k], s = source[p], as
 * sshdp_moe_gather_mxfp8 writes it (`dy` in `dtype`, `out` in MXFP8), and
 *   dweights[t][j] = sum over columns of dout[t] * y[place[t][j]]
 * in float32, 0 for dropped slots.  Either may be left out: dy and out NULL (source
 * and offsets are then not read), or dweights NULL (y and place are then not read).
 * The residual's gradient is dout itself.  Errors: as for the two calls above, ARG
 * also for no output at all. */
typedef struct {
  const void *dout, *y;
  const float *weights;
  const int32_t *place, *source, *offsets;
  void *dy;
  sshdp_mx_out out;
  float *dweights;
  int64_t tokens, rows, cols, ld_dout;
  int32_t top_k, experts, dtype, pad_;
} sshdp_moe_combine_grad;
int sshdp_moe_combine_backward(const sshdp_moe_combine_grad *args, void *stream);

/* MXFP8 products grouped by expert: the rows of A that sshdp_moe_sort gave expert e
 * (offsets[e] .. offsets[e + 1] - 1) with that expert's own matrix of the bank B,
 * whose rows are the experts' one after the other (groups equal parts: a bank
 * region of a plan, by sshdp_plan_mx_matrix).  Padding rows are rows like others.
 *   SSHDP_GEMM_NT: out[p][n] = sum_k A[p][k] B_e[n][k] (+ addend[p][n]);
 *   SSHDP_GEMM_NN: out[p][n] = sum_k A[p][k] B_e[k][n] (+ addend[p][n]),  B in
 *     BLOCK32X32: the input gradient, from the forward product's own codes;
 *   SSHDP_GEMM_TN: out_e[m][n] = sum over e's rows p of A[m][p] B[n][p] (+ addend):
 *     the weight gradients, groups x A.rows rows of float32.  A and B are the
 *     transposed operands of the two sides (codes_t, scales_t), the sorted rows
 *     along their columns; offsets must be multiples of 32.  An expert without rows
 *     gets its addend, or zeros.
 * Types and arithmetic are those of sshdp_gemm_mxfp8, except that NT with few rows an
 * expert (a rule on the sizes) has float32 sums for bfloat16 output too: a row's
 * bfloat16 result may differ between batches of different sizes, by the 8-bit
 * products' cut.  A's scales (TN: both) are ROWMAJOR, B's in any layout.  `addend`
 * (NULL for none) has out's type, shape and ld, and may be out; for bfloat16 it is
 * added in float32 ahead of the rounding.
 * `offsets`, groups + 1 device integers, may be NULL with one group, which then
 * has all rows.  Rows outside every expert's (behind the last one) are neither
 * read nor written; offsets that run backwards or past the rows make the call
 * write a part of out, never memory outside it.  No workspace.
 * Errors: ARG (null pointer, bad op, layout or dtype, groups < 1, no offsets for
 * several groups, TN with bfloat16), SCHEMA (the operands' K differ or are 0 or
 * over 2^22; B.rows not groups equal parts, of multiples of 32 in layouts that
 * group 32 rows; A's layout; NN without BLOCK32X32, of experts of under 4 blocks or
 * with B.cols over 2^23; TN with columns not a multiple of 128; ld_out < N; groups
 * over 1024; more than 2^22 tiles of 128 x 128), ALIGN (codes, addend, out;
 * offsets 4); HIP. */
enum { SSHDP_GEMM_TN = 2 };
int sshdp_gemm_mxfp8_grouped(const sshdp_mx_matrix *a, const sshdp_mx_matrix *b, int32_t op, const int32_t *offsets,
                             int32_t groups, const void *addend, void *out, int32_t out_dtype, int64_t ld_out,
                             void *stream);

/* The gated pair of products of an expert's (or, with one group, a dense) MLP, the
 * activation and G in one pass:
 *   gate = A Bg_e^T,  up = A Bu_e^T,  h = silu(gate) * up,
 *   silu(x) = x / (1 + exp(-x)),  codes, scales = G(h) along the rows (ROWMAJOR).
 * The products are sshdp_gemm_mxfp8's of bfloat16 output, every code under every scale:
 * each 8 consecutive k's are cut off at 2^-14 of the binade of their largest (few rows
 * an expert, a rule on the sizes: float32 sums, so a row's results may differ between
 * batches of different sizes by that cut).  Of normal operands with K = 2048 it moves
 * one code of h in 600, and one scale in 40000, that lies next to a rounding border;
 * there is no form with float32 sums for every size.  h is computed in float32
 * (within (1.25 |gate| + 8) 2^-24 of itself; for gates under -87.336, whose sigmoid is
 * no normal float32 number, within 2^-126 |gate up|) from the sums, before they are rounded.
 * `gate` and `up` (both or neither) receive the products in bfloat16, what the backward pass
 * needs; codes and scales may be left out then.  All outputs are dense, A.rows x N,
 * N = gate_w.rows / groups a multiple of 32; gate_w and up_w have the same shape
 * and layout.  The rest is as in sshdp_gemm_mxfp8_grouped with SSHDP_GEMM_NT. */
int sshdp_gemm_mxfp8_swiglu(const sshdp_mx_matrix *a, const sshdp_mx_matrix *gate_w, const sshdp_mx_matrix *up_w,
                            const int32_t *offsets, int32_t groups, uint8_t *codes, uint8_t *scales, void *gate,
                            void *up, void *stream);

/* The gated activation's gradient, with G behind: from gate and up (bfloat16, as
 * sshdp_gemm_mxfp8_swiglu leaves them) and dh, the gradient of h,
 *   s = 1 / (1 + exp(-gate)):  dgate = dh * up * s * (1 + gate * (1 - s)),
 *   dup = dh * gate * s,  and h = gate * s * up once more,
 * each in float32 (with s within (1.25 |gate| + 8) 2^-24 of itself) and then G along
 * the rows, along the columns (pitch `rows`, a multiple of 32 rows; zeros past a
 * block's last row in use), or both: the operands of the two input gradients, of the
 * weight gradients, and h along the tokens for the next projection's.  dh, gate and up are dense rows x cols.  Rows from offsets[groups]
 * on (offsets NULL: none) are neither read nor written.  Without dgate and dup, dh is
 * not read and may be NULL: the activation alone, of products kept in bfloat16.
 * s is 0 for gates under -87.336, where it is no normal float32 number.
 * Errors: ARG (null gate or up, dh missing, no output, half a pair, negative size,
 * groups < 1 with offsets), SCHEMA (cols not a multiple of 32, rows not one with an
 * output along columns, an edge over 2^30, groups over 1024), ALIGN (all but the
 * scales; offsets 4); HIP. */
typedef struct {
  const void *dh, *gate, *up;
  const int32_t *offsets;
  sshdp_mx_out dgate, dup, h;
  int64_t rows, cols;
  int32_t groups, pad_;
} sshdp_swiglu_grad;
int sshdp_swiglu_backward_mxfp8(const sshdp_swiglu_grad *args, void *stream);

/* Diagnostics.  The batched NT contraction used by Newton-Schulz, exposed to
 * test it alone: for b < batch, O[b] = bf16(alpha * P[b] Q[b]^T + beta * D[b])
 * with P[b] M x K, Q[b] N x K, O[b] M x N (bf16, row-major, dense, batch strides
 * M*K, N*K, M*N).  D is passed TRANSPOSED, DT[b] N x M (the layout in which the
 * update product reads X), or NULL (beta ignored); OT (optional) receives
 * O[b]^T (N x M).  M, N must be multiples of `tile` (128 or 256), K of 64.
 * tile 1281 / 2561: the same 128 / 256 tiles with both operands K-major (the
 * Gram read from X^T): P[b] K x M, Q[b] K x N row-major, M == N, D NULL.
 * Errors: ARG (null P, Q or O, non-positive sizes, unknown tile, K-major with D
 * or M != N), SCHEMA (sizes not multiples of the tile, or an operand panel that
 * one buffer resource cannot address: tile * K * 2 bytes, K-major
 * ((K - 1) * M + tile) * 2 bytes, at least 2^31), ALIGN. */
int sshdp_gemm_bf16_nt(const void *P, const void *Q, const void *D, void *O, void *OT, int32_t M,
                       int32_t N, int32_t K, int32_t batch, float alpha, float beta, int32_t tile,
                       void *stream);

/* Diagnostics.  What the Newton-Schulz tile schedule executed in the last
 * sshdp_update_muon / sshdp_update_step that used `workspace`: a unit whose
 * momentum was all zero has direction 0 and skips every product, so only the
 * other units count.  `units_per_group` (n_groups entries, or NULL) receives
 * each group's count of such units; `flops` (or NULL) the MFMA flops their
 * tiles executed in that step (stats.ns_tile_flops split per unit, summed over
 * them).  Reads the per-unit normalisation scales the call left in the
 * workspace: enqueues a copy on `stream` and synchronises with it.  Errors: ARG
 * (null plan, wrong device), STATE, WORKSPACE (null or smaller than
 * stats.workspace_bytes); HIP. */
int sshdp_ns_executed(const sshdp_plan *plan, const void *workspace, size_t workspace_bytes,
                      int32_t *units_per_group, double *flops, void *stream);

/* Per-stage kernel timing for benchmarking: when enabled on a plan, launching
 * calls bracket each kernel class with HIP events on the launch stream and
 * accumulate durations (milliseconds) and bracket counts; reading synchronises
 * on those events, returns the sums since the previous read and clears them.
 * Classes: 0 momentum (f0), 1 norm, 2 NS Gram, 3 NS poly,
 * 4 NS update (+f2), 5 AdamW, 6 AdamW+G fused, 7 G requant, 8 the whole
 * Newton-Schulz phase on the caller's stream (fork to join: NS launches of
 * different groups run concurrently on plan-owned streams, so classes 2-4 can
 * overlap in time), 9 G bf16 cast, and the Newton-Schulz launches of the
 * caller's stream alone (the groups whose sshdp_group_info.lane is 0): 10 Gram
 * and 11 poly (both tile sizes), 12 the update's 256-tile launch in the steps
 * before the last, 13 that launch in the last step (+f2).
 * Not thread-safe; for measurement only. */
enum { SSHDP_PROF_CLASSES = 14 };
int sshdp_profile_enable(sshdp_plan *plan, int32_t enable);
int sshdp_profile_read(sshdp_plan *plan, double *ms, int64_t *launches);

const char *sshdp_status_string(int code);
int sshdp_abi_version(void);

#ifdef __cplusplus
}
#endif
#endif /* SSHDP_H */
