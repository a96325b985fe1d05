"""Products with the experts' uncompressed weights, on torch tensors.

The rows of ``x``, ``y`` and their gradients are sorted by expert: expert e owns
rows ``expert_offsets[e] .. expert_offsets[e + 1] - 1`` (int32, on the device, as
``tileq_route`` leaves them).  Operands are bf16 or fp16, sums fp32, results
rounded once to ``out_dtype`` (the operands' type by default, or any of bf16,
fp16 and fp32)::

    y  = grouped_gemm(x, w, offsets)          # y[p]  = W_e x[p],    w [E, d_out, d_in]
    dx = grouped_gemm_dx(dy, w, offsets)      # dx[p] = W_e^T dy[p]
    dw = grouped_gemm_dw(x, dy, offsets)      # dW_e  = sum_p dy[p] x[p]^T

Rows outside the offsets' range belong to no expert: a given ``out`` keeps them,
a new one leaves them unset.  Calls are asynchronous on ``stream`` (the current
stream of the tensors' device by default), hold no state from one to the next
and can be captured into a CUDA graph.  Autograd does not record them: a backward
pass calls the gradients' products itself.  Tensors that do not fit raise
ValueError before anything is launched.
"""
from __future__ import annotations

import ctypes

import torch

from . import _lib as L

_CODE = {torch.bfloat16: L.TILEQ_DT_BF16, torch.float16: L.TILEQ_DT_F16, torch.float32: L.TILEQ_DT_F32}
_status_words: dict = {}


def _status_word(device: torch.device) -> torch.Tensor:
    """The device's status word, which the kernels write when a bounded wait gives up and never read."""
    ws = _status_words.get(device.index)
    if ws is None:
        if torch.cuda.is_current_stream_capturing():
            raise RuntimeError("make one call outside of the graph first: it allocates the device's status word")
        ws = torch.zeros(L.TILEQ_GROUPED_WS_BYTES, dtype=torch.uint8, device=device)
        torch.cuda.current_stream(device).synchronize()  # zeroed before a call on any other stream
        _status_words[device.index] = ws
    return ws


def expert_status(device="cuda") -> int:
    """Synchronously read and clear the first device error of these calls (0: none), as tileq_device_status."""
    device = torch.device(device)
    if device.index is None:
        device = torch.device(device.type, torch.cuda.current_device())
    with torch.cuda.device(device):
        torch.cuda.synchronize()
        return L.tileq_device_status(_status_word(device))


def _need(ok: bool, what: str):
    if not ok:
        raise ValueError(what)


def _rows(t: torch.Tensor, name: str, device=None, dtype=None) -> int:
    """The row stride of a [rows, cols] operand (0: contiguous)."""
    _need(t.dim() == 2 and t.is_cuda, f"{name} must be a 2-D CUDA tensor")
    _need(device is None or t.device == device, f"{name} is on another device")
    _need(dtype is None or t.dtype == dtype, f"{name} must be {dtype}")
    _need(t.shape[1] > 0, f"{name} has no columns")
    _need(t.stride(1) == 1 or t.shape[1] == 1 or t.shape[0] == 0, f"{name} must be contiguous in its last dimension")
    if t.shape[0] <= 1:
        return 0
    _need(t.stride(0) >= t.shape[1], f"{name} has overlapping rows")
    return t.stride(0)


def _weights(t: torch.Tensor, name: str, device, dtype=None):
    """(row stride, expert stride) of [E, d_out, d_in] weights."""
    _need(t.dim() == 3 and t.is_cuda, f"{name} must be a 3-D CUDA tensor [E, d_out, d_in]")
    _need(t.device == device, f"{name} is on another device")
    _need(dtype is None or t.dtype == dtype, f"{name} must be {dtype}")
    E, O, I = t.shape
    _need(1 <= E <= L.TILEQ_GROUPED_MAX_E and O > 0 and I > 0, f"{name}: 1 to {L.TILEQ_GROUPED_MAX_E} experts, no empty widths")
    _need(t.stride(2) == 1 or I == 1, f"{name} must be contiguous in its last dimension")
    ld = t.stride(1) if O > 1 else I
    _need(ld >= I and (E == 1 or t.stride(0) >= (O - 1) * ld + I), f"{name} has overlapping rows")
    return ld, (t.stride(0) if E > 1 else 0)


def _offsets(t, E: int, device):
    _need(t.dim() == 1 and t.shape[0] == E + 1 and t.dtype == torch.int32 and t.device == device and t.is_contiguous(),
          f"expert_offsets must be a contiguous int32 tensor of {E + 1} values on the operands' device")
    return t


def _code(dtype, default):
    dtype = default if dtype is None else dtype
    _need(dtype in _CODE, "out_dtype must be bfloat16, float16 or float32")
    return dtype


class _Call:
    """The stream of a call, with its device current; new outputs belong to that stream."""

    def __init__(self, device, stream):
        self.device, self.stream = device, stream
        self.ctx = None
        if isinstance(stream, int):
            self.stream = torch.cuda.ExternalStream(stream, device=device)
        if self.stream is not None:
            self.ctx = torch.cuda.stream(self.stream)
        elif torch.cuda.current_device() != device.index:
            self.ctx = torch.cuda.device(device)

    def __enter__(self):
        if self.ctx is not None:
            self.ctx.__enter__()
        return torch.cuda.current_stream(self.device).cuda_stream

    def __exit__(self, *exc):
        if self.ctx is not None:
            self.ctx.__exit__(*exc)
        return False


def _out(out, shape, dtype, device, name="out"):
    if out is None:
        return torch.empty(shape, dtype=dtype, device=device)
    _need(tuple(out.shape) == tuple(shape), f"{name} must have shape {tuple(shape)}")
    _need(out.dtype == dtype and out.device == device, f"{name} must be {dtype} on {device}")
    return out


def _operand(t, name):
    _need(t.dtype in (torch.bfloat16, torch.float16), f"{name} must be bfloat16 or float16")


def grouped_gemm(x, w, expert_offsets, out=None, out_dtype=None, stream=None):
    """y [P, d_out] with y[p] = W_e x[p]: x [P, d_in], w [E, d_out, d_in]."""
    _operand(x, "x")
    ld_x = _rows(x, "x")
    dev = x.device
    ld_w, stride_w = _weights(w, "w", dev, x.dtype)
    P, I = x.shape
    E, O, Iw = w.shape
    _need(I == Iw, f"x has {I} columns, w expects {Iw}")
    off = _offsets(expert_offsets, E, dev)
    dt = _code(out_dtype if out_dtype is not None else (out.dtype if out is not None else None), x.dtype)
    with _Call(dev, stream) as st:
        y = _out(out, (P, O), dt, dev)
        g = L.tileq_grouped(_CODE[x.dtype], _CODE[dt], E, P, I, O, ld_x, _rows(y, "out"), ld_w, stride_w, off.data_ptr())
        L.tileq_grouped_gemm(g, x, w, y, _status_word(dev), st)
    return y


def grouped_gemm_dx(dy, w, expert_offsets, out=None, out_dtype=None, stream=None):
    """dx [P, d_in] with dx[p] = W_e^T dy[p]: dy [P, d_out], w [E, d_out, d_in]."""
    _operand(dy, "dy")
    ld_y = _rows(dy, "dy")
    dev = dy.device
    ld_w, stride_w = _weights(w, "w", dev, dy.dtype)
    P, O = dy.shape
    E, Ow, I = w.shape
    _need(O == Ow, f"dy has {O} columns, w expects {Ow}")
    off = _offsets(expert_offsets, E, dev)
    dt = _code(out_dtype if out_dtype is not None else (out.dtype if out is not None else None), dy.dtype)
    with _Call(dev, stream) as st:
        dx = _out(out, (P, I), dt, dev)
        g = L.tileq_grouped(_CODE[dy.dtype], _CODE[dt], E, P, I, O, _rows(dx, "out"), ld_y, ld_w, stride_w, off.data_ptr())
        L.tileq_grouped_gemm_dx(g, dy, w, dx, _status_word(dev), st)
    return dx


def grouped_gemm_dw(x, dy, expert_offsets, out=None, out_dtype=None, stream=None):
    """dW [E, d_out, d_in] with dW_e = sum over the rows p of e of dy[p] x[p]^T, zeros for an expert without rows."""
    _operand(x, "x")
    ld_x = _rows(x, "x")
    dev = x.device
    ld_y = _rows(dy, "dy", dev, x.dtype)
    _need(x.shape[0] == dy.shape[0], "x and dy must have the same number of rows")
    (P, I), O = x.shape, dy.shape[1]
    E = expert_offsets.shape[0] - 1 if expert_offsets.dim() == 1 else 0
    _need(1 <= E <= L.TILEQ_GROUPED_MAX_E, f"expert_offsets must hold 2 to {L.TILEQ_GROUPED_MAX_E + 1} values")
    off = _offsets(expert_offsets, E, dev)
    dt = _code(out_dtype if out_dtype is not None else (out.dtype if out is not None else None), x.dtype)
    with _Call(dev, stream) as st:
        dw = _out(out, (E, O, I), dt, dev)
        ld_w, stride_w = _weights(dw, "out", dev)
        g = L.tileq_grouped(_CODE[x.dtype], _CODE[dt], E, P, I, O, ld_x, ld_y, ld_w, stride_w, off.data_ptr())
        L.tileq_grouped_gemm_dw(g, x, dy, dw, _status_word(dev), st)
    return dw
