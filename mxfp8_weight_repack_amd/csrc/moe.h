// moe.h -- launchers of the expert layer's operators.
#pragma once
#include "grouped_shape.h"
#include "internal.h"

namespace sshdp {

constexpr int kMoeMaxExperts = 1024;
constexpr int kMoeMaxTopK = 64;
constexpr int64_t kMoeMaxSlots = 1 << 24;

// Slots sorted by expert (k_moe.hip).  counts: moe_sort_counts(slots, experts) ints of workspace.
struct MoeSort {
  const void *ids;
  int64_t slots, rows;
  int32_t experts, align;
  int32_t *offsets, *place, *source;
  bool i64;
};
int64_t moe_sort_counts(int64_t slots, int experts);
hipError_t launch_moe_sort(const MoeSort &a, int32_t *counts, hipStream_t s);

// Rows gathered, weighted and quantised: sshdp_moe_gather's fields.
hipError_t launch_moe_gather(const sshdp_moe_gather &a, hipStream_t s);
hipError_t launch_moe_combine(const sshdp_moe_combine_args &a, hipStream_t s);
hipError_t launch_moe_dweights(const sshdp_moe_combine_grad &a, hipStream_t s);

// The gated activation and its gradient (k_act.hip): sshdp_swiglu_grad's fields.
hipError_t launch_swiglu_grad(const sshdp_swiglu_grad &a, hipStream_t s);

// Products grouped by expert (k_gemm_grouped.hip).  rows: all of A's (ROWS_*), n and k as in
// GemmMx, those of one expert's product.
struct GemmGrouped {
  GroupForm form;
  bool bf16;                          // output type
  GemmMx p;                           // m: rows of A; kColumns: k is all rows, m and n of one expert
  const uint8_t *b2, *b2s;            // kRowsGated
  uint16_t *gate, *up;                // kRowsGated, or NULL
  uint8_t *codes, *scales;            // kRowsGated, or NULL
  const uint16_t *addend16;           // bfloat16 output
  const int32_t *offsets;             // NULL: one group of all rows
  int32_t groups;
};
hipError_t launch_gemm_grouped(const GemmGrouped &g, hipStream_t s);

}  // namespace sshdp
