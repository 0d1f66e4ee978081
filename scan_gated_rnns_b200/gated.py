"""Torch-facing wrappers of the gated linear recurrence (argument marshalling
only; every operation runs in ``libsgr.so``):

    gated_scan(f, v, h0, cu_seqlens)     whole sequences, (B, T, D) or packed rows
    gated_scan_backward(...)             its gradients
    gated_scan_fn(f, v, h0, cu_seqlens)  the same, differentiable
    gated_step(f, v, state, slots)       one token per request, states in a pool

    gate="sigmoid":  a_t = sigmoid(f_t),      h_t = a_t h_{t-1} + (1 - a_t) v_t
    gate="log":      a_t = exp(min(f_t, 0)),  h_t = a_t h_{t-1} + v_t
"""
from __future__ import annotations

import functools
from typing import NamedTuple, Optional, Tuple

import torch
from torch.autograd.function import once_differentiable

from . import _abi, ops
from ._abi import check, lib

_DT = {torch.float32: _abi.SGR_F32, torch.bfloat16: _abi.SGR_BF16, torch.float16: _abi.SGR_F16}
_GATES = {"sigmoid": _abi.SGR_GATE_SIGMOID, "log": _abi.SGR_GATE_LOG}
_INDEX = {torch.int32: 4, torch.int64: 8}


def _gate(gate: str) -> int:
    try:
        return _GATES[gate]
    except (KeyError, TypeError):
        raise ValueError(f"gate must be 'sigmoid' or 'log', got {gate!r}") from None


def _dtype_code(t: torch.Tensor, name: str) -> int:
    try:
        return _DT[t.dtype]
    except KeyError:
        raise TypeError(f"{name}: dtype {t.dtype} is not supported (float32, bfloat16 or float16)") from None


def _dense(t: torch.Tensor) -> torch.Tensor:
    """An empty result of t's shape with dense rows (t's own may overlap)."""
    return torch.empty_like(t, memory_format=torch.contiguous_format)


# the raw handle of a device's current stream (a step is short beside the
# objects that the public call builds)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _launch(fn, device: int, *args) -> int:
    """fn(*args, stream) on `device` and its current stream."""
    stream = _raw_stream(device) if _raw_stream is not None else torch.cuda.current_stream(device).cuda_stream
    if device == torch.cuda.current_device():
        return fn(*args, stream)
    with torch.cuda.device(device):
        return fn(*args, stream)


def _row_stride(t: torch.Tensor, name: str) -> int:
    """Row stride, in elements, of a tensor whose leading dimensions count rows
    that lie evenly spaced, each of them contiguous."""
    shape, stride = t.shape, t.stride()
    if stride[-1] != 1 and shape[-1] > 1:
        raise ValueError(f"{name} must be contiguous along its last dimension")
    if len(shape) == 2:
        return stride[0] if shape[0] != 1 else shape[1]
    step, rows = None, 1
    for n, s in zip(reversed(shape[:-1]), reversed(stride[:-1])):
        if n == 1:
            continue
        if step is None:
            step = s
        elif s != step * rows and t.numel():
            raise ValueError(f"{name}: its leading dimensions must flatten to evenly spaced rows (make it contiguous)")
        rows *= n
    return shape[-1] if step is None else step


def _operand(t: torch.Tensor, like: Optional[torch.Tensor], name: str) -> int:
    ops._need_cuda(t, name)
    if like is not None and (t.shape != like.shape or t.dtype is not like.dtype or t.get_device() != like.get_device()):
        raise ValueError(f"{name} must match the first operand's shape, dtype and device")
    return _row_stride(t, name)


def _sequences(fn: str, f: torch.Tensor, cu: Optional[torch.Tensor]) -> Tuple[int, int, int, int, int]:
    """(rows, D, sequences, pointer of the bounds, bytes of one)."""
    if cu is None:
        if f.dim() == 3:
            return f.shape[0] * f.shape[1], f.shape[2], f.shape[0], 0, 0
        if f.dim() == 2:
            return f.shape[0], f.shape[1], 1, 0, 0
        raise ValueError(f"{fn}: f must be (B, T, D) or (T, D), got shape {tuple(f.shape)}")
    if f.dim() != 2:
        raise ValueError(f"{fn}: with cu_seqlens f must be packed rows (N, D), got shape {tuple(f.shape)}")
    ops._need_cuda(cu, fn + ": cu_seqlens")
    if cu.dtype not in _INDEX or cu.dim() != 1 or cu.shape[0] < 1 or not cu.is_contiguous() or \
            cu.get_device() != f.get_device():
        raise ValueError(f"{fn}: cu_seqlens must be a contiguous (sequences + 1,) int32 or int64 vector on {f.device}")
    return f.shape[0], f.shape[1], cu.shape[0] - 1, cu.data_ptr(), _INDEX[cu.dtype]


def _states(t: Optional[torch.Tensor], n: int, D: int, like: torch.Tensor, name: str, shared: bool) -> Tuple[int, int]:
    """(pointer, row stride) of fp32 states (n, D), or (D,) where one may serve
    all, on like's device."""
    if t is None:
        return 0, 0
    ops._need_cuda(t, name)
    if t.dtype is not torch.float32 or t.get_device() != like.get_device():
        raise ValueError(f"{name} must be float32 on {like.device}")
    shape, stride = t.shape, t.stride()
    if shared and len(shape) == 1:
        if shape[0] != D or (D > 1 and stride[0] != 1):
            raise ValueError(f"{name} must be a contiguous (D,) vector")
        return t.data_ptr(), 0
    if len(shape) != 2 or shape[0] != n or shape[1] != D or (D > 1 and stride[1] != 1):
        raise ValueError(f"{name} must be ({n}, {D}) with contiguous rows, got {tuple(shape)}")
    return t.data_ptr(), (stride[0] if n > 1 else D)


@functools.lru_cache(maxsize=4096)
def _sizes(rows: int, D: int) -> Tuple[int, int]:
    """(bytes of workspace, rows of kept states)."""
    return int(lib().sgr_gated_workspace_size(rows, D)), int(lib().sgr_gated_chunks(rows))


def _scratch(need: int, device, workspace: Optional[ops.Workspace]) -> Optional[torch.Tensor]:
    """The workspace given, or the call's own: of the caching allocator, so that
    calls on other streams and captured graphs each have theirs."""
    if workspace is None or not need:
        return torch.empty(need, dtype=torch.uint8, device=device) if need else None
    if workspace.nbytes < need or workspace.buf.device != device:
        raise ValueError(f"workspace must hold {need} bytes on {device}")
    return workspace.buf


class _Call(NamedTuple):
    """What a scan's arguments come to, beside their pointers."""
    gate: int
    dtype: int
    f_rs: int
    v_rs: int
    rows: int
    D: int
    n: int
    cu_bytes: int
    need: int        # bytes of workspace
    chunks: int      # rows of kept states


def _call(fn: str, f: torch.Tensor, v: torch.Tensor, cu: Optional[torch.Tensor], gate: str) -> _Call:
    g = _gate(gate)
    f_rs = _operand(f, None, fn + ": f")
    v_rs = _operand(v, f, fn + ": v")
    dt = _dtype_code(f, fn)
    rows, D, n, _, cb = _sequences(fn, f, cu)
    return _Call(g, dt, f_rs, v_rs, rows, D, n, cb, *_sizes(rows, D))


def _forward(c: _Call, f, v, hp, hss, cu, out, o_rs, zero, save_states, workspace=None):
    device = f.device
    h_last = torch.empty((c.n, c.D), dtype=torch.float32, device=device)
    states = torch.empty((c.chunks, c.D), dtype=torch.float32, device=device) if save_states else None
    ws = _scratch(c.need, device, workspace)
    code = _launch(lib().gated_scan, device.index, f.data_ptr(), c.f_rs, v.data_ptr(), c.v_rs, hp, hss,
                   cu.data_ptr() if c.cu_bytes else 0, c.cu_bytes, c.n, out.data_ptr(), o_rs, h_last.data_ptr(),
                   states.data_ptr() if save_states else 0, c.rows, c.D, c.gate, c.dtype, zero,
                   ws.data_ptr() if c.need else 0, c.need)
    check("gated_scan", code)
    return h_last, states


def _backward(c: _Call, f, v, hp, hss, cu, states, dh, dh_rs, lp, want_dh0, workspace=None):
    device = f.device
    df, dv = _dense(f), _dense(f)
    dh0 = torch.empty((c.n, c.D), dtype=torch.float32, device=device) if want_dh0 else None
    ws = _scratch(c.need, device, workspace)
    code = _launch(lib().gated_scan_backward, device.index, f.data_ptr(), c.f_rs, v.data_ptr(), c.v_rs, hp, hss,
                   cu.data_ptr() if c.cu_bytes else 0, c.cu_bytes, c.n, states.data_ptr(), dh.data_ptr(), dh_rs, lp,
                   df.data_ptr(), c.D, dv.data_ptr(), c.D, dh0.data_ptr() if want_dh0 else 0, c.rows, c.D, c.gate,
                   c.dtype, ws.data_ptr() if c.need else 0, c.need)
    check("gated_scan_backward", code)
    return df, dv, dh0


def gated_scan(f: torch.Tensor, v: torch.Tensor, h0: Optional[torch.Tensor] = None,
               cu_seqlens: Optional[torch.Tensor] = None, gate: str = "sigmoid",
               out: Optional[torch.Tensor] = None, save_states: bool = False,
               workspace: Optional[ops.Workspace] = None):
    """(h, h_last): the gated linear recurrence over f, v, (B, T, D) or, with
    cu_seqlens, packed rows (N, D); float32, bfloat16 or float16, rows of any
    even spacing (the halves of one projection are read in place).

    cu_seqlens: (S + 1,) ascending row bounds on the GPU; sequences may be
    empty, and rows outside [cu[0], cu[-1]) are padding: 0 in the result, left
    as they were in a given ``out``.  h0: float32 (S, D), or (D,) for every
    sequence.  h_last: float32 (S, D), the state behind each sequence.  With
    save_states a third result: what gated_scan_backward starts from.

    A wait between blocks that runs out leaves NaN.  With a workspace of
    workspace_size("gated", ...) bytes, which only one call at a time may use
    and only scans of this kind, its status() then says so; without one each
    call takes its own."""
    fn = "gated_scan"
    c = _call(fn, f, v, cu_seqlens, gate)
    hp, hss = _states(h0, c.n, c.D, f, fn + ": h0", True)
    zero, o_rs = out is None, c.D
    if zero:
        out = _dense(f)
    else:
        o_rs = _operand(out, f, fn + ": out")
    h_last, states = _forward(c, f, v, hp, hss, cu_seqlens, out, o_rs, int(zero), save_states,
                              workspace)
    return (out, h_last, states) if save_states else (out, h_last)


def gated_scan_backward(f: torch.Tensor, v: torch.Tensor, h0: Optional[torch.Tensor], states: torch.Tensor,
                        dh: torch.Tensor, dh_last: Optional[torch.Tensor] = None,
                        cu_seqlens: Optional[torch.Tensor] = None, gate: str = "sigmoid", want_dh0: bool = True,
                        workspace: Optional[ops.Workspace] = None):
    """(df, dv, dh0) for dL/dh = dh and dL/dh_last = dh_last through
    h, h_last, states = gated_scan(f, v, h0, cu_seqlens, gate, save_states=True);
    dh0 is float32 (S, D), one row per sequence (None unless want_dh0).  workspace
    as for gated_scan."""
    fn = "gated_scan_backward"
    c = _call(fn, f, v, cu_seqlens, gate)
    dh_rs = _operand(dh, f, fn + ": dh")
    hp, hss = _states(h0, c.n, c.D, f, fn + ": h0", True)
    lp, lss = _states(dh_last, c.n, c.D, f, fn + ": dh_last", False)
    if lp and c.n > 1 and lss != c.D:
        raise ValueError(f"{fn}: dh_last must be contiguous")
    _, sss = _states(states, c.chunks, c.D, f, fn + ": states", False)
    if states is None or (c.chunks > 1 and sss != c.D):
        raise ValueError(f"{fn}: states must be the contiguous ({c.chunks}, {c.D}) tensor that gated_scan saved")
    return _backward(c, f, v, hp, hss, cu_seqlens, states, dh, dh_rs, lp, want_dh0, workspace)


class GatedScan(torch.autograd.Function):
    """The states inside the sequences are kept for the backward pass (about
    one float32 row per 96 rows); the outputs are not."""

    @staticmethod
    def forward(ctx, f, v, h0, cu_seqlens, gate):
        c = _call("gated_scan", f, v, cu_seqlens, gate)
        hp, hss = _states(h0, c.n, c.D, f, "gated_scan: h0", True)
        h = _dense(f)
        h_last, states = _forward(c, f, v, hp, hss, cu_seqlens, h, c.D, 1, True)
        ctx.save_for_backward(f, v, h0, cu_seqlens, states)
        ctx.call = c
        ctx.set_materialize_grads(False)
        return h, h_last

    @staticmethod
    @once_differentiable
    def backward(ctx, dh, dh_last):
        f, v, h0, cu_seqlens, states = ctx.saved_tensors
        if dh is None and dh_last is None:
            return None, None, None, None, None
        # hooks on saved tensors may have laid them out anew
        c = ctx.call._replace(f_rs=_row_stride(f, "f"), v_rs=_row_stride(v, "v"))
        hp, hss = _states(h0, c.n, c.D, f, "h0", True)
        dh = torch.zeros_like(f, memory_format=torch.contiguous_format) if dh is None else dh.contiguous()
        last = None if dh_last is None else dh_last.contiguous()
        df, dv, dh0 = _backward(c, f, v, hp, hss, cu_seqlens, states.contiguous(), dh, c.D,
                                last.data_ptr() if last is not None else 0, ctx.needs_input_grad[2])
        if dh0 is not None and h0.dim() == 1:
            dh0 = dh0.sum(0)
        return df, dv, dh0, None, None


def gated_scan_fn(f: torch.Tensor, v: torch.Tensor, h0: Optional[torch.Tensor] = None,
                  cu_seqlens: Optional[torch.Tensor] = None, gate: str = "sigmoid"):
    """(h, h_last) of gated_scan with gradients for f, v and h0, from either
    result (first derivatives only).  In a CUDA graph capture forward and
    backward together, on leaves that no graph built outside the capture still
    holds: PyTorch cannot capture a backward pass that reaches back to one."""
    return GatedScan.apply(f, v, h0, cu_seqlens, gate)


def gated_step(f: torch.Tensor, v: torch.Tensor, state: torch.Tensor, slots: Optional[torch.Tensor] = None,
               gate: str = "sigmoid", out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """h (M, D): one token of the recurrence for each of M requests; f, v (M, D)
    rows, state the float32 pool (slots, D), updated in place.

    slots: (M,) int32 or int64 on the GPU, the pool row of each request (None:
    row i).  A slot outside the pool marks a padding row: 0 in the result, left
    as it was in a given ``out``.  A slot named by several rows takes their
    tokens in row order.  Every row looks through all slots: meant for batches
    of up to some thousand requests."""
    fn = "gated_step"
    g = _gate(gate)
    f_rs = _operand(f, None, "gated_step: f")
    if f.dim() != 2:
        raise ValueError(f"{fn}: f must be (M, D), got shape {tuple(f.shape)}")
    v_rs = _operand(v, f, "gated_step: v")
    dt = _dtype_code(f, fn)
    M, D = f.shape
    n_slots = state.shape[0] if state.dim() == 2 else 0
    if state.dim() != 2 or state.shape[1] != D:
        raise ValueError(f"{fn}: state must be (slots, {D}), got {tuple(state.shape)}")
    sp, srs = _states(state, n_slots, D, f, "gated_step: state", False)
    device = f.get_device()
    kp = kb = 0
    if slots is not None:
        ops._need_cuda(slots, "gated_step: slots")
        if slots.dtype not in _INDEX or slots.dim() != 1 or slots.shape[0] != M or not slots.is_contiguous() or \
                slots.get_device() != device:
            raise ValueError(f"{fn}: slots must be a contiguous ({M},) int32 or int64 vector on {f.device}")
        kp, kb = slots.data_ptr(), _INDEX[slots.dtype]
    elif n_slots < M:
        raise ValueError(f"{fn}: state has {n_slots} rows for {M} requests")
    zero, o_rs = out is None, D
    if zero:
        out = _dense(f)
    else:
        o_rs = _operand(out, f, "gated_step: out")
    code = _launch(lib().gated_step, device, f.data_ptr(), f_rs, v.data_ptr(), v_rs, sp, srs, n_slots, kp, kb,
                   out.data_ptr(), o_rs, M, D, g, dt, zero)
    if code:
        check(fn, code)
    return out
