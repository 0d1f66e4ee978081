"""Torch-facing wrappers of the 8-bit projection (argument marshalling only;
both operations run in ``libsgr.so``):

    q, scale = int8_quantize(x)                       rows of x in 8 bits
    y = int8_projection(x, w_q, w_scale, ...)         s_x s_w (q_x w_q^T) + bias
"""
from __future__ import annotations

import functools
from typing import Optional, Tuple

import torch

from . import _abi, ops
from ._abi import check, lib
from .gated import _DT, _dtype_code, _launch, _row_stride


def int8_quantize(x: torch.Tensor) -> Tuple[torch.Tensor, torch.Tensor]:
    """(q, scale) of x (..., K), float32, bfloat16 or float16: q int8 (..., K)
    and scale float32 (...), scale = largest |x| of the row times the float32
    1/127 (at least 2^-100) and q = x / scale to the nearest whole number, ties to even.  The
    rows of q start on 16-byte boundaries, as the tensor-core projection takes
    them, for tokens and for a weight matrix's channels alike."""
    fn = "int8_quantize"
    ops._need_cuda(x, fn + ": x")
    if x.dim() < 1:
        raise ValueError(f"{fn}: x must have at least one dimension")
    dt = _dtype_code(x, fn)
    x_rs = _row_stride(x, fn + ": x")
    K = x.shape[-1]
    lead = x.shape[:-1]
    rows = lead.numel()
    pad = -(-K // 16) * 16
    buf = torch.empty((*lead, pad), dtype=torch.int8, device=x.device)
    q = buf[..., :K]
    scale = torch.empty(lead, dtype=torch.float32, device=x.device)
    code = _launch(lib().int8_quantize, x.get_device(), x.data_ptr(), x_rs, q.data_ptr(), pad, scale.data_ptr(), rows, K, dt)
    check(fn, code)
    return q, scale


@functools.lru_cache(maxsize=4096)
def _workspace(rows: int, K: int, dtype: int) -> int:
    return int(lib().sgr_int8_workspace_size(rows, K, dtype))


def _vector(t: Optional[torch.Tensor], shape, like: torch.Tensor, name: str) -> int:
    if t is None:
        return 0
    ops._need_cuda(t, name)
    if t.dtype is not torch.float32 or t.shape != shape or not t.is_contiguous() or t.get_device() != like.get_device():
        raise ValueError(f"{name} must be a contiguous float32 {tuple(shape)} tensor on {like.device}")
    return t.data_ptr()


def int8_projection(x: torch.Tensor, w_q: torch.Tensor, w_scale: torch.Tensor, x_scale: Optional[torch.Tensor] = None,
                    bias: Optional[torch.Tensor] = None, out_dtype: Optional[torch.dtype] = None,
                    out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """y (..., N) = x_scale w_scale (x w_q^T) + bias, the sum exact in int32.

    x (..., K): int8 with x_scale (...), or float32, bfloat16 or float16, whose
    rows are quantised as by int8_quantize within the call.  w_q (N, K) int8
    with w_scale (N,) (int8_quantize of the weights); bias float32 (N,).
    out_dtype: float32, bfloat16 or float16; by default x's own, float32 for
    int8 x.  K is at most 2^17 - 1."""
    fn = "int8_projection"
    ops._need_cuda(x, fn + ": x")
    ops._need_cuda(w_q, fn + ": w_q")
    if x.dim() < 1:
        raise ValueError(f"{fn}: x must have at least one dimension")
    quantised = x.dtype == torch.int8
    if quantised != (x_scale is not None):
        raise ValueError(f"{fn}: x_scale goes with int8 x, and only with it")
    xdt = _abi.SGR_I8 if quantised else _dtype_code(x, fn + ": x")
    if w_q.dtype != torch.int8 or w_q.dim() != 2 or w_q.shape[1] != x.shape[-1] or \
            w_q.get_device() != x.get_device():
        raise ValueError(f"{fn}: w_q must be int8 (N, {x.shape[-1]}) on {x.device}")
    N, K = w_q.shape
    if K < 1:
        raise ValueError(f"{fn}: x needs at least one column")
    lead = x.shape[:-1]
    rows = lead.numel()
    x_rs = _row_stride(x, fn + ": x")
    w_rs = _row_stride(w_q, fn + ": w_q")
    sp = _vector(x_scale, lead, x, fn + ": x_scale")
    wp = _vector(w_scale, (N,), x, fn + ": w_scale")
    bp = _vector(bias, (N,), x, fn + ": bias")
    if out is None:
        if out_dtype is None:
            out_dtype = torch.float32 if quantised else x.dtype
        if out_dtype not in _DT:
            raise TypeError(f"{fn}: out_dtype {out_dtype} is not supported (float32, bfloat16 or float16)")
        out = torch.empty((*lead, N), dtype=out_dtype, device=x.device)
    else:
        ops._need_cuda(out, fn + ": out")
        if tuple(out.shape) != (*lead, N) or out.get_device() != x.get_device() or out_dtype not in (None, out.dtype):
            raise ValueError(f"{fn}: out must be {(*lead, N)} of out_dtype on {x.device}")
    ydt = _dtype_code(out, fn + ": out")
    y_rs = _row_stride(out, fn + ": out")
    need = 0 if quantised else _workspace(rows, K, xdt)
    ws = torch.empty(need, dtype=torch.uint8, device=x.device) if need else None
    code = _launch(lib().int8_projection, x.get_device(), x.data_ptr(), x_rs, xdt, sp, w_q.data_ptr(), w_rs, wp, bp,
                   out.data_ptr(), y_rs, ydt, rows, K, N, ws.data_ptr() if need else 0, need)
    check(fn, code)
    return out
