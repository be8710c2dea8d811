"""One MI355X's share of the SS-HSDP update phase: Muon (momentum, batched bf16
MFMA Newton-Schulz, weight update), AdamW and in-place MXFP8 requantisation
of packed fp32 roots, as hand-written HIP for gfx950 behind the C ABI in
include/sshdp.h, and the operators around it: gradient norm and clipping, MXFP8
quantisation, residual RMS norm, MXFP8 products, and a mixture-of-experts layer.  This package is the thin ctypes binding of that library.
"""

from ._lib import (  # noqa: F401
    LIB_PATH, SshdpError, Plan, buffers, muon_hp, adamw_hp, update_muon, update_adamw, requant_mxfp8,
    cast_bf16, rs_reduce, rs_accumulate,
    grad_workspace, grad_sumsq, grad_clip, grad_clip_norm, quant_mxfp8,
    rmsnorm_mxfp8, rmsnorm_backward, rmsnorm_backward_workspace, mx_matrix, gemm_mxfp8, gemm_mxfp8_workspace,
    mx_pair, moe_rows, moe_sort, moe_sort_workspace, moe_gather_mxfp8, moe_combine, moe_combine_backward,
    gemm_mxfp8_grouped, gemm_mxfp8_swiglu, swiglu_backward_mxfp8,
    update_step, update_step_noalloc, gemm_bf16_nt, lib, PROF_CLASSES, ERROR_NAMES, NOALLOC_SCRATCH_BYTES,
)
