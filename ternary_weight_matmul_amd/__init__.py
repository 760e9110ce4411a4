"""Ternary-weight matmul for AMD MI355X (gfx950): thin Python binding of libtern.so.

Every step of the computation runs in the HIP kernels behind the C ABI of
``include/tern.h``; this module only marshals arguments (device pointers,
sizes, dtype codes and the current HIP stream).  PyTorch supplies device
memory and streams.  If ``libtern.so`` has not been built, importing the
library raises: there is no fallback implementation.

    import ternary_weight_matmul_amd as tern
    packed = tern.pack(T)                     # int8 [N,K] in {-1,0,1} -> uint8 [N,K/4]
    T2 = tern.unpack(packed, K)               # uint8 [N,K/4] -> int8 [N,K]
    y = tern.matmul(x, packed, scales, out_dtype=torch.bfloat16)

    codes, exps = tern.mx_quantize(w)         # [N,K] -> 4-bit floats, a power-of-two scale per 32
    y = tern.mx_matmul(x, codes, exps)        # x . w^T, x in 16 bits
    y = tern.mx_matmul_mx(*tern.mx_quantize(x), codes, exps)    # both in 4 bits
    y = tern.moe(x, logits, gate_up, gate_up_scales, down, down_scales, top_k=8)    # ternary experts
"""
from __future__ import annotations

from ._lib import (  # noqa: F401
    DTYPE_CODE,
    PATH_AUTO,
    PATH_GEMV,
    PATH_MFMA,
    STATUS,
    TernError,
    lib,
    library_path,
)
from .ops import (block_map, dequant, matmul, matmul_blockmap, matmul_blockmap_into, matmul_into,  # noqa: F401
                  matmul_s8, matmul_s8_into, moe, moe_into, mx_dequant, mx_matmul, mx_matmul_into, mx_matmul_mx,
                  mx_matmul_mx_into, mx_quantize, pack, quantize_scales, shard_columns, shard_k, stream_copy, unpack)

GROUP = 128
MX_BLOCK = 32
GEMV_MAX_M = 4
