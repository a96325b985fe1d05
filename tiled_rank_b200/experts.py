"""Products with the experts' uncompressed weights, on torch tensors.

The rows of ``x``, ``y`` and their gradients are sorted by expert: expert e owns
rows ``expert_offsets[e] .. expert_offsets[e + 1] - 1`` (int32, on the device, as
``tileq_route`` leaves them).  Operands are bf16 or fp16, sums fp32, results
rounded once to ``out_dtype`` (the operands' type by default, or any of bf16,
fp16 and fp32)::

    y  = grouped_gemm(x, w, offsets)          # y[p]  = W_e x[p],    w [E, d_out, d_in]
    dx = grouped_gemm_dx(dy, w, offsets)      # dx[p] = W_e^T dy[p]
    dw = grouped_gemm_dw(x, dy, offsets)      # dW_e  = sum_p dy[p] x[p]^T

In 8 bits, with e4m3 values and an fp32 scale for every 128 columns of a row and
every 128 x 128 block of a weight matrix::

    wq, ws = fp8_quantize_weights(w)                              # once
    xq, xs = fp8_quantize(x, rows=rows)                           # gathers row rows[p] of x for row p
    gu = fp8_gemm(xq, xs, wq, ws, offsets)                        # gate and up in one product
    hq, hs = fp8_quantize(gu, swiglu=True, row_scale=weight)      # silu(gate) * up * weight
    y = fp8_gemm(hq, hs, wdq, wds, offsets)

The quantisers' scales are powers of two (the smallest that bring the block's
largest magnitude to 448 or less); the product takes any scales.  With a 2-D wq
the product is dense.

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


def _quantised(q, shape, device):
    """A new e4m3 tensor whose rows start at multiples of 16 bytes, as the product reads them, or the given one."""
    if q is None:
        q = torch.empty((*shape[:-1], -(-shape[-1] // 16) * 16), dtype=torch.float8_e4m3fn, device=device)
        return q if q.shape[-1] == shape[-1] else q[..., :shape[-1]]
    return _out(q, shape, torch.float8_e4m3fn, device)


def _scales(s, shape, device, name="scales"):
    if s is None:
        return torch.empty(shape, dtype=torch.float32, device=device)
    _need(tuple(s.shape) == tuple(shape) and s.dtype == torch.float32 and s.device == device and s.stride(-1) == 1,
          f"{name} must be a float32 tensor {tuple(shape)} on {device}, contiguous in its last dimension")
    _need(s.dim() > 2 or s.shape[0] <= 1 or s.stride(0) >= s.shape[1], f"{name} has overlapping rows")
    return s


def _vector(t, n: int, dtype, name: str, device):
    if t is None:
        return None
    _need(t.dim() == 1 and t.shape[0] == n and t.dtype == dtype and t.device == device and t.is_contiguous(),
          f"{name} must be a contiguous {dtype} tensor of {n} values on the operands' device")
    return t.data_ptr()


def fp8_quantize(x, rows=None, swiglu=False, row_scale=None, out=None, scales=None, stream=None):
    """Rows in e4m3 with a scale for every 128 columns: (q [R, C], scales [ceil(C / 128), R]).

    x [T, C] (swiglu: [T, 2C], gate then up, of which silu(gate) * up is quantised) in bf16, fp16
    or fp32.  rows: int32 [R], the row of x of each row of q (outside [0, T): zeros); without it
    R = T.  row_scale: fp32 [R], a factor of each row of q.
    """
    _need(x.dtype in _CODE, "x must be bfloat16, float16 or float32")
    ld_x, dev = _rows(x, "x"), x.device
    T, C = x.shape
    if swiglu:
        _need(C % 2 == 0, "x must hold the gate's and the up projection's columns")
        C //= 2
    R = T if rows is None else rows.numel()
    at = _vector(rows, R, torch.int32, "rows", dev)
    factor = _vector(row_scale, R, torch.float32, "row_scale", dev)
    with _Call(dev, stream) as st:
        q = _quantised(out, (R, C), dev)
        s = _scales(scales, (-(-C // 128), R), dev)
        a = L.tileq_fp8_rows(_CODE[x.dtype], R, T, C, int(bool(swiglu)), at, factor, ld_x, _rows(q, "out"),
                             s.stride(0) if s.shape[0] > 1 else 0)
        L.tileq_fp8_quantize(a, x, q, s, st)
    return q, s


def fp8_quantize_weights(w, out=None, scales=None, stream=None):
    """Weights [E, d_out, d_in] (or one expert's [d_out, d_in]) in e4m3 with a scale for every 128 x 128 block:
    (q like w, scales [E, ceil(d_out / 128), ceil(d_in / 128)], without E for one)."""
    _need(w.dtype in _CODE, "w must be bfloat16, float16 or float32")
    if w.dim() == 2:
        q, s = fp8_quantize_weights(w[None], None if out is None else out[None], None if scales is None else scales[None],
                                    stream)
        return q[0], s[0]
    dev = w.device
    ld_w, stride_w = _weights(w, "w", dev)
    E, O, I = w.shape
    with _Call(dev, stream) as st:
        q = _quantised(out, (E, O, I), dev)
        ld_q, stride_q = _weights(q, "out", dev)
        s = _scales(scales, (E, -(-O // 128), -(-I // 128)), dev)
        _need(s.is_contiguous(), "scales must be contiguous")
        g = L.tileq_grouped(_CODE[w.dtype], 0, E, 0, I, O, 0, 0, ld_w, stride_w, None)
        L.tileq_fp8_quantize_weights(g, w, q, ld_q, stride_q, s, st)
    return q, s


def fp8_gemm(xq, xs, wq, ws, expert_offsets=None, out=None, out_dtype=None, stream=None):
    """y [P, d_out] (bf16, or out_dtype) from e4m3 rows xq [P, d_in] with scales xs [ceil(d_in / 128), P]
    and e4m3 weights wq [E, d_out, d_in] with scales ws [E, ceil(d_out / 128), ceil(d_in / 128)].

    Dense, without expert_offsets: wq [d_out, d_in], ws [ceil(d_out / 128), ceil(d_in / 128)].
    """
    if wq.dim() == 2:
        _need(expert_offsets is None, "a 2-D wq is one expert's, for all rows: no expert_offsets")
        wq, ws = wq[None], ws[None]
    else:
        _need(expert_offsets is not None, "expert_offsets say which rows are whose")
    f8 = torch.float8_e4m3fn
    _need(xq.dtype == f8, "xq must be float8_e4m3fn")
    ld_x, dev = _rows(xq, "xq"), xq.device
    ld_w, stride_w = _weights(wq, "wq", dev, f8)
    P, I = xq.shape
    E, O, Iw = wq.shape
    _need(I == Iw, f"xq has {I} columns, wq expects {Iw}")
    kb = -(-I // 128)
    _scales(xs, (kb, P), dev, "xs")
    _scales(ws, (E, -(-O // 128), kb), dev, "ws")
    _need(ws.is_contiguous(), "ws must be contiguous")
    off = None if expert_offsets is None else _offsets(expert_offsets, E, dev).data_ptr()
    dt = _code(out_dtype if out_dtype is not None else (out.dtype if out is not None else None), torch.bfloat16)
    with _Call(dev, stream) as st:
        y = _out(out, (P, O), dt, dev)
        g = L.tileq_grouped(L.TILEQ_DT_E4M3, _CODE[dt], E, P, I, O, ld_x, _rows(y, "out"), ld_w, stride_w, off)
        L.tileq_fp8_gemm(g, xq, xs, xs.stride(0) if kb > 1 else 0, wq, ws, y, _status_word(dev), st)
    return y
