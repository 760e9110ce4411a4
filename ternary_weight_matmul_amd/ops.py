"""Torch-tensor entry points over the C ABI (argument marshalling only).

Each function checks what only the binding can check (tensor device, dtype,
contiguity), passes raw device pointers, sizes and the current HIP stream to
the library, and raises TernError on a non-OK status.  The library itself
validates shapes, group, alignment and dtypes before launching anything.
"""
from __future__ import annotations

from typing import Optional

import torch

from ._lib import (DTYPE_CODE, PATH_AUTO, PATH_GEMV, PATH_GEMV_B16, PATH_GEMV_FP4, PATH_GEMV_MFMA, PATH_MFMA,
                   TernError, lib)

_TORCH_CODE = {torch.float16: DTYPE_CODE["f16"], torch.bfloat16: DTYPE_CODE["bf16"],
               torch.float32: DTYPE_CODE["f32"]}
_PATHS = {"auto": PATH_AUTO, "gemv": PATH_GEMV, "mfma": PATH_MFMA, "gemv_mfma": PATH_GEMV_MFMA,
          "gemv_fp4": PATH_GEMV_FP4, "gemv_b16": PATH_GEMV_B16}


def _stream(t: torch.Tensor) -> int:
    return torch.cuda.current_stream(t.device).cuda_stream


def _need(t: torch.Tensor, name: str, dtype: torch.dtype, ndim: int = 2) -> None:
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != ndim:
        raise ValueError(f"{name} must be {ndim}-D, got shape {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous (reshape to 2-D and call .contiguous())")


def _check(status: int, where: str) -> None:
    if status != 0:
        raise TernError(status, where)


def pack(T: torch.Tensor, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """int8 [N,K] (values -1/0/+1) -> uint8 [N,K/4], 2 bits per weight."""
    _need(T, "T", torch.int8)
    N, K = T.shape
    if out is None:
        out = torch.empty((N, K // 4), dtype=torch.uint8, device=T.device)
    _need(out, "out", torch.uint8)
    if tuple(out.shape) != (N, K // 4):
        raise ValueError("out must be [N, K/4]")
    _check(lib.tern_pack(T.data_ptr(), out.data_ptr(), N, K, _stream(T)), "tern_pack")
    return out


def unpack(packed: torch.Tensor, K: int, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """uint8 [N,K/4] -> int8 [N,K] in {-1,0,+1}."""
    _need(packed, "packed", torch.uint8)
    N = packed.shape[0]
    if packed.shape[1] * 4 != K:
        raise ValueError(f"packed has {packed.shape[1]} bytes per row, K={K} needs {K // 4}")
    if out is None:
        out = torch.empty((N, K), dtype=torch.int8, device=packed.device)
    _need(out, "out", torch.int8)
    _check(lib.tern_unpack(packed.data_ptr(), out.data_ptr(), N, K, _stream(packed)), "tern_unpack")
    return out


def matmul_into(x: torch.Tensor, packed: torch.Tensor, scales: torch.Tensor, out: torch.Tensor,
                group: int = 128, path: str = "auto") -> torch.Tensor:
    """out[M,N] = x[M,K] . (T*S)^T; x fp16/bf16, scales fp16 [N,K/group]."""
    if x.dtype not in (torch.float16, torch.bfloat16):
        raise TypeError("x must be float16 or bfloat16")
    _need(x, "x", x.dtype)
    _need(packed, "packed", torch.uint8)
    _need(scales, "scales", torch.float16)
    if out.dtype not in _TORCH_CODE:
        raise TypeError("out must be float32, bfloat16 or float16")
    _need(out, "out", out.dtype)
    M, K = x.shape
    N = packed.shape[0]
    if packed.shape[1] * 4 != K or tuple(scales.shape) != (N, K // group if group > 0 else 0) \
            or tuple(out.shape) != (M, N):
        raise ValueError(f"shape mismatch: x {tuple(x.shape)}, packed {tuple(packed.shape)}, "
                         f"scales {tuple(scales.shape)}, out {tuple(out.shape)}")
    st = lib.tern_matmul_path(x.data_ptr(), _TORCH_CODE[x.dtype], packed.data_ptr(), scales.data_ptr(),
                              out.data_ptr(), _TORCH_CODE[out.dtype], M, N, K, group, _PATHS[path],
                              _stream(x))
    _check(st, "tern_matmul")
    return out


def matmul(x: torch.Tensor, packed: torch.Tensor, scales: torch.Tensor,
           out_dtype: torch.dtype = torch.bfloat16, group: int = 128, path: str = "auto") -> torch.Tensor:
    """Y[M,N] = x[M,K] . (T*S)^T with fp32 accumulation; returns a new tensor."""
    out = torch.empty((x.shape[0], packed.shape[0]), dtype=out_dtype, device=x.device)
    return matmul_into(x, packed, scales, out, group, path)


def dequant(packed: torch.Tensor, scales: torch.Tensor, out_dtype: torch.dtype = torch.float16,
            group: int = 128, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Dense W[N,K] = t * s (the pages' dequantise-then-GEMM comparison route)."""
    _need(packed, "packed", torch.uint8)
    _need(scales, "scales", torch.float16)
    N = packed.shape[0]
    K = packed.shape[1] * 4
    if out is None:
        out = torch.empty((N, K), dtype=out_dtype, device=packed.device)
    if out.dtype not in (torch.float16, torch.bfloat16):
        raise TypeError("out must be float16 or bfloat16")
    _need(out, "out", out.dtype)
    if tuple(out.shape) != (N, K) or (group > 0 and tuple(scales.shape) != (N, K // group)):
        raise ValueError("shape mismatch")
    _check(lib.tern_dequant(packed.data_ptr(), scales.data_ptr(), out.data_ptr(), _TORCH_CODE[out.dtype],
                            N, K, group, _stream(packed)), "tern_dequant")
    return out


# --- zero-block skipping -----------------------------------------------------

def block_map(packed: torch.Tensor, group: int = 128) -> torch.Tensor:
    """packed [N,K/4] -> int32 [N, ceil(K/group/32)], the bits of tern_block_map (stored as int32)."""
    _need(packed, "packed", torch.uint8)
    N = packed.shape[0]
    K = packed.shape[1] * 4
    words = (K // group + 31) // 32
    out = torch.empty((N, words), dtype=torch.int32, device=packed.device)
    _check(lib.tern_block_map(packed.data_ptr(), out.data_ptr(), N, K, group, _stream(packed)),
           "tern_block_map")
    return out


def matmul_blockmap_into(x: torch.Tensor, packed: torch.Tensor, scales: torch.Tensor, bmap: torch.Tensor,
                         out: torch.Tensor, group: int = 128) -> torch.Tensor:
    """matmul_into that skips the blocks `bmap` (from block_map) leaves unmarked."""
    if x.dtype not in (torch.float16, torch.bfloat16):
        raise TypeError("x must be float16 or bfloat16")
    _need(x, "x", x.dtype)
    _need(packed, "packed", torch.uint8)
    _need(scales, "scales", torch.float16)
    _need(bmap, "bmap", torch.int32)
    if out.dtype not in _TORCH_CODE:
        raise TypeError("out must be float32, bfloat16 or float16")
    _need(out, "out", out.dtype)
    M, K = x.shape
    N = packed.shape[0]
    words = (K // group + 31) // 32 if group > 0 else 0
    if packed.shape[1] * 4 != K or tuple(scales.shape) != (N, K // group if group > 0 else 0) \
            or tuple(bmap.shape) != (N, words) or tuple(out.shape) != (M, N):
        raise ValueError(f"shape mismatch: x {tuple(x.shape)}, packed {tuple(packed.shape)}, "
                         f"scales {tuple(scales.shape)}, bmap {tuple(bmap.shape)}, out {tuple(out.shape)}")
    st = lib.tern_matmul_blockmap(x.data_ptr(), _TORCH_CODE[x.dtype], packed.data_ptr(), scales.data_ptr(),
                                  bmap.data_ptr(), out.data_ptr(), _TORCH_CODE[out.dtype], M, N, K, group,
                                  _stream(x))
    _check(st, "tern_matmul_blockmap")
    return out


def matmul_blockmap(x: torch.Tensor, packed: torch.Tensor, scales: torch.Tensor, bmap: torch.Tensor,
                    out_dtype: torch.dtype = torch.bfloat16, group: int = 128) -> torch.Tensor:
    out = torch.empty((x.shape[0], packed.shape[0]), dtype=out_dtype, device=x.device)
    return matmul_blockmap_into(x, packed, scales, bmap, out, group)


# --- int8 block scales -------------------------------------------------------

def quantize_scales(scales: torch.Tensor, group: int = 128):
    """fp16 scales [N,G] -> (int8 codes [N,G], fp32 row factors [N]); scale = q * r."""
    _need(scales, "scales", torch.float16)
    N, G = scales.shape
    q = torch.empty((N, G), dtype=torch.int8, device=scales.device)
    r = torch.empty((N,), dtype=torch.float32, device=scales.device)
    _check(lib.tern_quantize_scales(scales.data_ptr(), q.data_ptr(), r.data_ptr(), N, G * group, group,
                                    _stream(scales)), "tern_quantize_scales")
    return q, r


def matmul_s8_into(x: torch.Tensor, packed: torch.Tensor, scales_q: torch.Tensor, row_factor: torch.Tensor,
                   out: torch.Tensor, group: int = 128, path: str = "auto") -> torch.Tensor:
    """out[M,N] = x . (T * (q * r))^T with int8 block codes q [N,K/group] and row factors r [N]."""
    if x.dtype not in (torch.float16, torch.bfloat16):
        raise TypeError("x must be float16 or bfloat16")
    _need(x, "x", x.dtype)
    _need(packed, "packed", torch.uint8)
    _need(scales_q, "scales_q", torch.int8)
    _need(row_factor, "row_factor", torch.float32, ndim=1)
    if out.dtype not in _TORCH_CODE:
        raise TypeError("out must be float32, bfloat16 or float16")
    _need(out, "out", out.dtype)
    M, K = x.shape
    N = packed.shape[0]
    if packed.shape[1] * 4 != K or tuple(scales_q.shape) != (N, K // group if group > 0 else 0) \
            or tuple(row_factor.shape) != (N,) or tuple(out.shape) != (M, N):
        raise ValueError(f"shape mismatch: x {tuple(x.shape)}, packed {tuple(packed.shape)}, "
                         f"scales_q {tuple(scales_q.shape)}, row_factor {tuple(row_factor.shape)}, "
                         f"out {tuple(out.shape)}")
    st = lib.tern_matmul_s8(x.data_ptr(), _TORCH_CODE[x.dtype], packed.data_ptr(), scales_q.data_ptr(),
                            row_factor.data_ptr(), out.data_ptr(), _TORCH_CODE[out.dtype], M, N, K, group,
                            _PATHS[path], _stream(x))
    _check(st, "tern_matmul_s8")
    return out


def matmul_s8(x: torch.Tensor, packed: torch.Tensor, scales_q: torch.Tensor, row_factor: torch.Tensor,
              out_dtype: torch.dtype = torch.bfloat16, group: int = 128, path: str = "auto") -> torch.Tensor:
    out = torch.empty((x.shape[0], packed.shape[0]), dtype=out_dtype, device=x.device)
    return matmul_s8_into(x, packed, scales_q, row_factor, out, group, path)


# --- microscaled 4-bit floats ---------------------------------------------------
#
# A decode step calls these once per layer with microseconds of GPU work, so
# the binding's own time counts: the checks are single expressions, and the
# stream and the device are read through the raw accessors (0.1 us each where
# torch.cuda.current_stream and torch.cuda.device take 2.0 and 1.4).

_FLOAT16S = (torch.float16, torch.bfloat16)
_FLOATS = tuple(_TORCH_CODE)


def _launch(fn, where: str, t: torch.Tensor, *args) -> None:
    """fn(*args, stream) on t's device and its current stream."""
    index = t.get_device()
    if index == torch._C._cuda_getDevice():
        status = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    else:
        with torch.cuda.device(index):
            status = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    if status != 0:
        raise TernError(status, where)


def _need_at(t: torch.Tensor, name: str, index: int, dtypes, shape) -> None:
    """t lies on GPU `index` (which is one), dense, with one of the types and the shape."""
    if t.get_device() == index and t.dtype in dtypes and t.shape == shape and t.is_contiguous():
        return
    if t.get_device() != index:
        raise ValueError(f"{name} must be on the device of the other tensors, cuda:{index}; it is on {t.device}")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be one of {', '.join(str(d) for d in dtypes)}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have the shape {tuple(shape)}, got {tuple(t.shape)}")
    raise ValueError(f"{name} must be contiguous (call .contiguous())")


def _need_matrix(t: torch.Tensor, name: str, dtypes) -> int:
    """t is a dense matrix of one of the types on a GPU, whose index is returned."""
    index = t.get_device()
    if index >= 0 and t.dtype in dtypes and t.dim() == 2 and t.is_contiguous():
        return index
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be one of {', '.join(str(d) for d in dtypes)}, got {t.dtype}")
    _need(t, name, t.dtype)
    return index


_U8 = (torch.uint8,)
_F16 = (torch.float16,)


def _need_codes(codes: torch.Tensor, exps: torch.Tensor, index: int, prefix: str = ""):
    """(rows, K) of a matrix held as codes and exps on GPU `index`."""
    at = _need_matrix(codes, prefix + "codes", _U8)
    rows, half = codes.shape
    if half % 16 != 0:
        raise ValueError(f"{prefix}codes must be [R, K/2] with K a multiple of 32, got {tuple(codes.shape)}")
    if at != index:
        _need_at(codes, prefix + "codes", index, _U8, codes.shape)
    _need_at(exps, prefix + "exps", index, _U8, (rows, half // 16))
    return rows, 2 * half


def mx_quantize(x: torch.Tensor):
    """x [M,K] fp16/bf16/fp32 -> (codes uint8 [M,K/2], exps uint8 [M,K/32]): e2m1 values with a
    power-of-two scale per 32, rounded to nearest even (tern_mx_quantize)."""
    _need_matrix(x, "x", _FLOATS)
    M, K = x.shape
    codes = x.new_empty((M, K // 2), dtype=torch.uint8)
    exps = x.new_empty((M, K // 32), dtype=torch.uint8)
    _launch(lib.tern_mx_quantize, "tern_mx_quantize", x, x.data_ptr(), _TORCH_CODE[x.dtype], codes.data_ptr(),
            exps.data_ptr(), M, K)
    return codes, exps


def mx_dequant(codes: torch.Tensor, exps: torch.Tensor, out_dtype: torch.dtype = torch.float32,
               out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The values [M,K] of a matrix held as codes and exps; exact in fp32 and bf16."""
    M, K = _need_codes(codes, exps, codes.get_device())
    if out is None:
        if out_dtype not in _TORCH_CODE:
            raise TypeError("out_dtype must be float32, bfloat16 or float16")
        out = torch.empty((M, K), dtype=out_dtype, device=codes.device)
    else:
        _need_at(out, "out", codes.get_device(), _FLOATS, (M, K))
    _launch(lib.tern_mx_dequant, "tern_mx_dequant", codes, codes.data_ptr(), exps.data_ptr(), out.data_ptr(),
            _TORCH_CODE[out.dtype], M, K)
    return out


def mx_matmul_into(x: torch.Tensor, codes: torch.Tensor, exps: torch.Tensor, out: torch.Tensor) -> torch.Tensor:
    """out[M,N] = x[M,K] . W^T, x fp16/bf16, W [N,K] held as codes and exps."""
    index = _need_matrix(x, "x", _FLOAT16S)
    N, K = _need_codes(codes, exps, index)
    M, KX = x.shape
    if KX != K:
        raise ValueError(f"shape mismatch: x {tuple(x.shape)}, codes {tuple(codes.shape)}")
    _need_at(out, "out", index, _FLOATS, (M, N))
    _launch(lib.tern_mx_matmul, "tern_mx_matmul", x, x.data_ptr(), _TORCH_CODE[x.dtype], codes.data_ptr(),
            exps.data_ptr(), out.data_ptr(), _TORCH_CODE[out.dtype], M, N, K)
    return out


def mx_matmul(x: torch.Tensor, codes: torch.Tensor, exps: torch.Tensor,
              out_dtype: torch.dtype = torch.bfloat16) -> torch.Tensor:
    """Y[M,N] = x[M,K] . W^T with fp32 accumulation, W [N,K] held as codes and exps; returns a new tensor."""
    out = x.new_empty((x.shape[0], codes.shape[0]), dtype=out_dtype)
    return mx_matmul_into(x, codes, exps, out)


def mx_matmul_mx_into(x_codes: torch.Tensor, x_exps: torch.Tensor, codes: torch.Tensor, exps: torch.Tensor,
                      out: torch.Tensor) -> torch.Tensor:
    """out[M,N] = X . W^T with both matrices held as codes and exps."""
    index = x_codes.get_device()
    M, K = _need_codes(x_codes, x_exps, index, "x_")
    N, KW = _need_codes(codes, exps, index)
    if K != KW:
        raise ValueError(f"shape mismatch: x_codes {tuple(x_codes.shape)}, codes {tuple(codes.shape)}")
    _need_at(out, "out", index, _FLOATS, (M, N))
    _launch(lib.tern_mx_matmul_mx, "tern_mx_matmul_mx", x_codes, x_codes.data_ptr(), x_exps.data_ptr(),
            codes.data_ptr(), exps.data_ptr(), out.data_ptr(), _TORCH_CODE[out.dtype], M, N, K)
    return out


def mx_matmul_mx(x_codes: torch.Tensor, x_exps: torch.Tensor, codes: torch.Tensor, exps: torch.Tensor,
                 out_dtype: torch.dtype = torch.bfloat16) -> torch.Tensor:
    """Y[M,N] = X . W^T with both matrices held as codes and exps; returns a new tensor."""
    out = x_codes.new_empty((x_codes.shape[0], codes.shape[0]), dtype=out_dtype)
    return mx_matmul_mx_into(x_codes, x_exps, codes, exps, out)


# --- mixture of ternary experts -------------------------------------------------

_F32 = (torch.float32,)
_I32 = (torch.int32,)


def _need_experts(x: torch.Tensor, gate_up: torch.Tensor, gate_up_scales: torch.Tensor, down: torch.Tensor,
                  down_scales: torch.Tensor, out: torch.Tensor, group: int):
    """(GPU index, T, E, H, F) of an expert layer's operands."""
    device = _need_matrix(x, "x", _FLOAT16S)
    if gate_up.dim() != 3 or down.dim() != 3:
        raise ValueError("gate_up must be [E, 2F, H/4] and down [E, H, F/4]")
    if group <= 0:
        raise ValueError("group must be positive")
    T, H = x.shape
    E, F = gate_up.shape[0], down.shape[2] * 4
    _need_at(gate_up, "gate_up", device, _U8, (E, 2 * F, H // 4))
    _need_at(gate_up_scales, "gate_up_scales", device, _F16, (E, 2 * F, H // group))
    _need_at(down, "down", device, _U8, (E, H, F // 4))
    _need_at(down_scales, "down_scales", device, _F16, (E, H, F // group))
    _need_at(out, "out", device, _FLOATS, (T, H))
    return device, T, E, H, F


def moe_into(x: torch.Tensor, logits: torch.Tensor, gate_up: torch.Tensor, gate_up_scales: torch.Tensor,
             down: torch.Tensor, down_scales: torch.Tensor, out: torch.Tensor, top_k: int,
             renormalize: bool = True, group: int = 128) -> torch.Tensor:
    """out [T,H] = the mixture-of-experts layer of tern_moe: x [T,H] fp16/bf16, logits [T,E],
    gate_up [E,2F,H/4] and down [E,H,F/4] packed codes, their fp16 scales one per 128."""
    device, T, E, H, F = _need_experts(x, gate_up, gate_up_scales, down, down_scales, out, group)
    _need_at(logits, "logits", device, _FLOATS, (T, E))
    nbytes = lib.tern_moe_workspace(T, E, top_k, H, F)
    # allocated on the current stream: torch's allocator keeps it for this call until that stream
    # has passed it, and inside a graph capture it belongs to the graph
    ws = x.new_empty((nbytes,), dtype=torch.uint8)
    _launch(lib.tern_moe, "tern_moe", x, x.data_ptr(), _TORCH_CODE[x.dtype], logits.data_ptr(),
            _TORCH_CODE[logits.dtype], gate_up.data_ptr(), gate_up_scales.data_ptr(), down.data_ptr(),
            down_scales.data_ptr(), out.data_ptr(), _TORCH_CODE[out.dtype], T, E, top_k, H, F, group,
            int(renormalize), ws.data_ptr(), nbytes)
    return out


def moe(x: torch.Tensor, logits: torch.Tensor, gate_up: torch.Tensor, gate_up_scales: torch.Tensor,
        down: torch.Tensor, down_scales: torch.Tensor, top_k: int, renormalize: bool = True,
        out_dtype: Optional[torch.dtype] = None, group: int = 128) -> torch.Tensor:
    """The layer's outputs [T,H] (of x's type unless out_dtype is given) as a new tensor.  With fp32
    outputs the hidden values keep all their bits, with 16-bit outputs 16 of them in less time."""
    out = x.new_empty(x.shape, dtype=out_dtype)
    return moe_into(x, logits, gate_up, gate_up_scales, down, down_scales, out, top_k, renormalize, group)


_SCORES = {"softmax": 0, "sigmoid": 1}


def moe_route(logits: torch.Tensor, top_k: int, score: str = "softmax", bias: Optional[torch.Tensor] = None,
              groups: int = 1, keep_groups: int = 1, group_best: int = 1, renormalize: bool = True, scale: float = 1.0):
    """The experts ids int32 [T,top_k] of every token and their weights fp32 [T,top_k] from logits [T,E]
    (tern_moe_route): softmax or sigmoid scores, chosen by score + bias (fp32 [E]) among the keep_groups of
    `groups` groups of consecutive experts whose group_best largest add up to the most.  Without a bias
    experts are chosen by their logits, and so are groups with group_best 1."""
    index = _need_matrix(logits, "logits", _FLOATS)
    T, E = logits.shape
    if score not in _SCORES:
        raise ValueError("score must be 'softmax' or 'sigmoid'")
    if bias is not None:
        _need_at(bias, "bias", index, _F32, (E,))
    if not 1 <= top_k <= max(E, 1):
        raise ValueError(f"top_k must be in [1, {E}], got {top_k}")
    ids = logits.new_empty((T, top_k), dtype=torch.int32)
    weights = logits.new_empty((T, top_k), dtype=torch.float32)
    _launch(lib.tern_moe_route, "tern_moe_route", logits, logits.data_ptr(), _TORCH_CODE[logits.dtype],
            bias.data_ptr() if bias is not None else 0, ids.data_ptr(), weights.data_ptr(), T, E, top_k, _SCORES[score],
            groups, keep_groups, group_best, int(renormalize), scale)
    return ids, weights


def moe_routed_into(x: torch.Tensor, ids: torch.Tensor, weights: torch.Tensor, gate_up: torch.Tensor,
                    gate_up_scales: torch.Tensor, down: torch.Tensor, down_scales: torch.Tensor, out: torch.Tensor,
                    group: int = 128) -> torch.Tensor:
    """out [T,H] = moe_into with the experts ids int32 [T,k] and their weights fp32 [T,k] given (from
    moe_route, or any router)."""
    device, T, E, H, F = _need_experts(x, gate_up, gate_up_scales, down, down_scales, out, group)
    if ids.dim() != 2:
        raise ValueError(f"ids must be [T, k], got {tuple(ids.shape)}")
    top_k = ids.shape[1]
    _need_at(ids, "ids", device, _I32, (T, top_k))
    _need_at(weights, "weights", device, _F32, (T, top_k))
    nbytes = lib.tern_moe_workspace(T, E, top_k, H, F)
    ws = x.new_empty((nbytes,), dtype=torch.uint8)   # as in moe_into
    _launch(lib.tern_moe_routed, "tern_moe_routed", x, x.data_ptr(), _TORCH_CODE[x.dtype], ids.data_ptr(),
            weights.data_ptr(), gate_up.data_ptr(), gate_up_scales.data_ptr(), down.data_ptr(), down_scales.data_ptr(),
            out.data_ptr(), _TORCH_CODE[out.dtype], T, E, top_k, H, F, group, ws.data_ptr(), nbytes)
    return out


def moe_routed(x: torch.Tensor, ids: torch.Tensor, weights: torch.Tensor, gate_up: torch.Tensor,
               gate_up_scales: torch.Tensor, down: torch.Tensor, down_scales: torch.Tensor,
               out_dtype: Optional[torch.dtype] = None, group: int = 128) -> torch.Tensor:
    """The layer's outputs [T,H] (of x's type unless out_dtype is given) as a new tensor."""
    out = x.new_empty(x.shape, dtype=out_dtype)
    return moe_routed_into(x, ids, weights, gate_up, gate_up_scales, down, down_scales, out, group)


# --- norms and 8-bit activations --------------------------------------------------

_I8 = (torch.int8,)


def _q_shape(M: int, K: int, group: int):
    """Shape of the scales of 8-bit activations [M,K]: one per row (group 0) or per `group` of a row."""
    if group not in (0, 128):
        raise ValueError("group must be 0 (a scale per row) or 128")
    if group and K % group != 0:
        raise ValueError(f"K = {K} must be a multiple of the group of 128")
    return (M, K // group) if group else (M, 1)


def _need_q8(codes: torch.Tensor, scales: torch.Tensor, index: int):
    """(M, K, group) of 8-bit activations held as codes [M,K] and scales [M,1] or [M,K/128] on GPU `index`."""
    _need_matrix(codes, "codes", _I8)
    M, K = codes.shape
    if scales.dim() != 2 or scales.shape[0] != M or not (scales.shape[1] == 1 or scales.shape[1] * 128 == K):
        raise ValueError(f"scales must be [M, 1] or [M, K/128] for codes {tuple(codes.shape)}, got {tuple(scales.shape)}")
    _need_at(scales, "scales", index, _F32, scales.shape)
    return M, K, 0 if scales.shape[1] == 1 else 128


def rms_norm_into(x: torch.Tensor, weight: Optional[torch.Tensor], out: Optional[torch.Tensor] = None,
                  codes: Optional[torch.Tensor] = None, scales: Optional[torch.Tensor] = None, eps: float = 1e-6,
                  residual: Optional[torch.Tensor] = None, residual_out: Optional[torch.Tensor] = None) -> None:
    """The norm of tern_rms_norm of x [M,K] into out [M,K], codes [M,K] with scales, or both.  With a
    residual [M,K] (x's type or fp32) the norm is that of x + residual, which goes to residual_out
    (residual itself if not given)."""
    index = _need_matrix(x, "x", _FLOATS)
    M, K = x.shape
    if out is None and codes is None:
        raise ValueError("out or codes must be given")
    if out is not None:
        _need_at(out, "out", index, _FLOATS, (M, K))
    group = 0
    if codes is not None:
        if scales is None:
            raise ValueError("scales must be given with codes")
        _need_at(codes, "codes", index, _I8, (M, K))
        group = _need_q8(codes, scales, index)[2]
    elif scales is not None:
        raise ValueError("codes must be given with scales")
    if residual is not None:
        residual_out = residual if residual_out is None else residual_out
        _need_at(residual_out, "residual_out", index, (residual.dtype,), (M, K))
    elif residual_out is not None:
        raise ValueError("residual must be given with residual_out")
    _rms_norm(x, index, M, K, weight, out, codes, scales, group, eps, residual, residual_out)


def _rms_norm(x, index, M, K, weight, out, codes, scales, group, eps, residual, residual_out) -> None:
    """The launch, of inputs yet to be checked (x aside) and outputs that are as they should be."""
    if weight is not None:
        _need_at(weight, "weight", index, _FLOATS, (K,))
    if residual is not None:
        _need_at(residual, "residual", index, (x.dtype, torch.float32), (M, K))
    _launch(lib.tern_rms_norm, "tern_rms_norm", x, x.data_ptr(), _TORCH_CODE[x.dtype],
            residual.data_ptr() if residual is not None else 0, _TORCH_CODE[residual.dtype] if residual is not None else 0,
            weight.data_ptr() if weight is not None else 0, _TORCH_CODE[weight.dtype] if weight is not None else 0,
            residual_out.data_ptr() if residual_out is not None else 0, out.data_ptr() if out is not None else 0,
            _TORCH_CODE[out.dtype] if out is not None else 0, codes.data_ptr() if codes is not None else 0,
            scales.data_ptr() if scales is not None else 0, group, M, K, eps)


def rms_norm(x: torch.Tensor, weight: Optional[torch.Tensor], eps: float = 1e-6,
             residual: Optional[torch.Tensor] = None, out_dtype: Optional[torch.dtype] = None):
    """y = h / sqrt(mean(h^2) + eps) * weight of every row, h = x [M,K]; y in x's type unless out_dtype is
    given.  With a residual [M,K] h is x + residual in the residual's type, and (y, h) is returned."""
    index = _need_matrix(x, "x", _FLOATS)
    M, K = x.shape
    if out_dtype is not None and out_dtype not in _FLOATS:
        raise TypeError("out_dtype must be float32, bfloat16 or float16")
    out = x.new_empty((M, K), dtype=out_dtype)
    h = None if residual is None else x.new_empty((M, K), dtype=residual.dtype)
    _rms_norm(x, index, M, K, weight, out, None, None, 0, eps, residual, h)
    return out if h is None else (out, h)


def rms_norm_q8(x: torch.Tensor, weight: Optional[torch.Tensor], eps: float = 1e-6,
                residual: Optional[torch.Tensor] = None, group: int = 0):
    """rms_norm with the outputs as 8-bit activations: (codes int8 [M,K], scales fp32 [M,1], or [M,K/128]
    with group 128), and h with a residual."""
    index = _need_matrix(x, "x", _FLOATS)
    M, K = x.shape
    codes = x.new_empty((M, K), dtype=torch.int8)
    scales = x.new_empty(_q_shape(M, K, group), dtype=torch.float32)
    h = None if residual is None else x.new_empty((M, K), dtype=residual.dtype)
    _rms_norm(x, index, M, K, weight, None, codes, scales, group, eps, residual, h)
    return (codes, scales) if h is None else (codes, scales, h)


def q8_quantize(x: torch.Tensor, group: int = 0):
    """x [M,K] -> 8-bit activations (codes int8 [M,K], scales fp32 [M,1], or [M,K/128] with group 128):
    127 x / a rounded to nearest even, a the largest magnitude of the row or block (tern_q8_quantize)."""
    _need_matrix(x, "x", _FLOATS)
    M, K = x.shape
    codes = x.new_empty((M, K), dtype=torch.int8)
    scales = x.new_empty(_q_shape(M, K, group), dtype=torch.float32)
    _launch(lib.tern_q8_quantize, "tern_q8_quantize", x, x.data_ptr(), _TORCH_CODE[x.dtype], codes.data_ptr(),
            scales.data_ptr(), group, M, K)
    return codes, scales


def q8_dequant(codes: torch.Tensor, scales: torch.Tensor, out_dtype: torch.dtype = torch.float32) -> torch.Tensor:
    """The values codes * scales of 8-bit activations as a new tensor."""
    M, K, group = _need_q8(codes, scales, codes.get_device())
    if out_dtype not in _TORCH_CODE:
        raise TypeError("out_dtype must be float32, bfloat16 or float16")
    out = codes.new_empty((M, K), dtype=out_dtype)
    _launch(lib.tern_q8_dequant, "tern_q8_dequant", codes, codes.data_ptr(), scales.data_ptr(), group, out.data_ptr(),
            _TORCH_CODE[out_dtype], M, K)
    return out


def matmul_q8_into(codes: torch.Tensor, scales: torch.Tensor, packed: torch.Tensor, weight_scales: torch.Tensor,
                   out: torch.Tensor, group: int = 128) -> torch.Tensor:
    """out[M,N] = X . (T*S)^T with X held as 8-bit activations, W as packed codes [N,K/4] and fp16 scales
    [N,K/group]."""
    index = codes.get_device()
    M, K, q_group = _need_q8(codes, scales, index)
    _need_at(out, "out", index, _FLOATS, (M, packed.shape[0]))
    return _matmul_q8(codes, scales, packed, weight_scales, out, index, M, K, q_group, group)


def _matmul_q8(codes, scales, packed, weight_scales, out, index, M, K, q_group, group) -> torch.Tensor:
    """The launch, of weights yet to be checked."""
    if group <= 0:
        raise ValueError("group must be positive")
    if packed.dim() != 2 or packed.shape[1] * 4 != K:
        raise ValueError(f"shape mismatch: codes {tuple(codes.shape)}, packed {tuple(packed.shape)}")
    N = packed.shape[0]
    _need_at(packed, "packed", index, _U8, (N, K // 4))
    _need_at(weight_scales, "weight_scales", index, _F16, (N, K // group))
    nbytes = lib.tern_matmul_q8_workspace(M, N, K) if M > 32 else 0
    ws = codes.new_empty((nbytes,)) if nbytes else None   # as in moe_into
    _launch(lib.tern_matmul_q8, "tern_matmul_q8", codes, codes.data_ptr(), scales.data_ptr(), q_group, packed.data_ptr(),
            weight_scales.data_ptr(), out.data_ptr(), _TORCH_CODE[out.dtype], M, N, K, group,
            ws.data_ptr() if nbytes else 0, nbytes)
    return out


def matmul_q8(codes: torch.Tensor, scales: torch.Tensor, packed: torch.Tensor, weight_scales: torch.Tensor,
              out_dtype: torch.dtype = torch.bfloat16, group: int = 128) -> torch.Tensor:
    """Y[M,N] = X . (T*S)^T with X held as 8-bit activations (from rms_norm_q8 or q8_quantize); a new tensor."""
    index = codes.get_device()
    M, K, q_group = _need_q8(codes, scales, index)
    if out_dtype not in _FLOATS:
        raise TypeError("out_dtype must be float32, bfloat16 or float16")
    out = codes.new_empty((M, packed.shape[0]), dtype=out_dtype)
    return _matmul_q8(codes, scales, packed, weight_scales, out, index, M, K, q_group, group)


# --- one GPU's share of a sharded layer (no communication here) -------------

def shard_columns(packed: torch.Tensor, scales: torch.Tensor, rank: int, world: int):
    """Column-parallel shard: whole rows n of W (output columns of Y).

    Rows [rank*N/world, (rank+1)*N/world) of the packed matrix and of the
    scales (2kiu.com/news/5082861 §5.1: a column split cuts the packed weight
    and its scale by output rows).  Row slices of row-major tensors are
    contiguous views: nothing is copied.
    """
    N = packed.shape[0]
    a, b = N * rank // world, N * (rank + 1) // world
    return packed[a:b], scales[a:b]


def shard_k(x: torch.Tensor, packed: torch.Tensor, scales: torch.Tensor, rank: int, world: int,
            group: int = 128):
    """Row-parallel shard: a K range cut on 128-weight block boundaries.

    The block boundaries keep every scale with its weights (§3.2, third check,
    and §5.1 of the same page: a K split must align with the blocks).  Returns
    contiguous copies of x[:, k0:k1], packed[:, k0/4:k1/4], scales[:, g0:g1];
    the partial products of all ranks sum to the full result.
    """
    K = x.shape[1]
    groups = K // group
    g0, g1 = groups * rank // world, groups * (rank + 1) // world
    k0, k1 = g0 * group, g1 * group
    return (x[:, k0:k1].contiguous(), packed[:, k0 // 4:k1 // 4].contiguous(),
            scales[:, g0:g1].contiguous())


def stream_copy(src: torch.Tensor, dst: Optional[torch.Tensor] = None, nbytes: Optional[int] = None) -> None:
    """Calibration only: stream ``nbytes`` bytes of ``src`` (all of it by default) and copy
    them into ``dst`` when given; with no ``dst`` the bytes are only read.  Device tensors,
    contiguous, 16-byte aligned; nbytes a multiple of 16."""
    if not src.is_cuda or not src.is_contiguous():
        raise ValueError("src must be a contiguous device tensor")
    n = src.numel() * src.element_size() if nbytes is None else int(nbytes)
    if n > src.numel() * src.element_size():
        raise ValueError("nbytes exceeds src")
    dptr = 0
    if dst is not None:
        if not dst.is_cuda or not dst.is_contiguous() or dst.numel() * dst.element_size() < n:
            raise ValueError("dst must be a contiguous device tensor of at least nbytes")
        dptr = dst.data_ptr()
    _check(lib.tern_stream_copy(src.data_ptr(), dptr, n, _stream(src)), "tern_stream_copy")
