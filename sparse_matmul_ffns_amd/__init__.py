"""MI355X (gfx950) semi-structured sparse FFN matmuls: N:M and V:N:M pruning,
compression and sparse x dense products, the mixture-of-experts FFN in 8-bit
floating point, and the dense FFN block around the products, behind the
libnmsparse C ABI.

The binding functions live in `sparse_matmul_ffns_amd.nmsparse`; the library
is loaded on first use and must have been built with
`python -m sparse_matmul_ffns_amd.build`.
"""

from .nmsparse import (  # noqa: F401
    NM_ERR_TOO_LARGE,
    NmError,
    fp8_gemm_nt,
    fp8_gemm_nt_grouped,
    fp8_gemm_nt_grouped_k,
    fp8_quantize,
    fp8_quantize_t,
    fp8_quantize_weight,
    grad_clip,
    grad_norm,
    lib,
    linear_bwd_act,
    linear_bwd_w,
    linear_bwd_x,
    linear_fwd,
    mfma_rate_probe,
    moe_combine,
    moe_combine_bwd,
    moe_plan,
    moe_plan_rows,
    moe_route,
    moe_route_bwd,
    nm_compress,
    nm_decompress,
    nm_prune,
    nm_prune_compress,
    nm_prune_compress_transpose,
    nm_reprune_t_transpose,
    nm_reprune_t_transpose_panels,
    nm_to_panels,
    nm_reprune_t,
    prune_act_venom,
    rms_norm,
    rms_norm_bwd,
    rms_norm_fp8,
    sddmm_nm,
    sizes,
    spmm_nm,
    spmm_nm_general,
    general_work_bytes,
    general_scratch_bytes,
    spmm_nm_general_noalloc,
    sddmm_venom,
    spmm_venom_tn,
    venom_tn_work_bytes,
    spmm_nm_t,
    spmm_nm_t_panels,
    spmm_nm_t_lowrank,
    spmm_nm_t_relu_venom,
    spmm_venom,
    transpose,
)
from .moe import ExpertFFN  # noqa: E402,F401
from .dense import DenseFFN  # noqa: E402,F401
