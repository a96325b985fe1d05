"""Products with the experts' uncompressed weights, on torch tensors.

The rows of ``x``, ``y`` and their gradients are sorted by expert: expert e owns
rows ``expert_offsets[e] .. expert_offsets[e + 1] - 1`` (int32, on the device, as
``tileq_route`` leaves them).  Operands are bf16 or fp16, sums fp32, results
rounded once to ``out_dtype`` (the operands' type by default, or any of bf16,
fp16 and fp32)::

    y  = grouped_gemm(x, w, offsets)          # y[p]  = W_e x[p],    w [E, d_out, d_in]
    dx = grouped_gemm_dx(dy, w, offsets)      # dx[p] = W_e^T dy[p]
    dw = grouped_gemm_dw(x, dy, offsets)      # dW_e  = sum_p dy[p] x[p]^T

With ``None`` for the offsets there is one expert, of every row.

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
stream of the tensors' device by default; the caller orders another one behind the
work that fills the tensors, and may drop them once the call has returned; a new
result belongs to ``stream``).  They hold no state from one to the next and can be
captured into a CUDA graph (after one call on that device outside of a graph, which
allocates its status word).

Autograd does not record them: a backward pass calls the gradients' products itself.
So that no gradient is lost unseen, a product with an operand that requires one raises
ValueError while gradients are enabled: make it under ``torch.no_grad()`` or in a
``torch.autograd.Function``.  (The quantisers take such tensors; their results are
steps, without a gradient.)  Tensors that do not fit raise ValueError, and TileQError
what the library refuses (a stride or an address that is no multiple of 16 bytes, a
result that shares memory with an operand), before anything is launched.
"""
from __future__ import annotations

from ctypes import byref

import torch

from . import _lib as L

_CODE = {torch.bfloat16: L.TILEQ_DT_BF16, torch.float16: L.TILEQ_DT_F16, torch.float32: L.TILEQ_DT_F32}
_OPERAND = {torch.bfloat16: L.TILEQ_DT_BF16, torch.float16: L.TILEQ_DT_F16}
_I32, _F32, _F8 = torch.int32, torch.float32, torch.float8_e4m3fn
_written = torch.autograd.graph.increment_version  # a given result: autograd knows that a tensor it saved has changed
_status_words: dict = {}   # of each device: the tensor and its address

# A small product takes the GPU a few microseconds, so what a call costs on the host counts: the checks below read each
# attribute once, compare devices by number (-1: not on a GPU) and build a message only when they raise.


def _status_word(index: int):
    """The device's status word, which the kernels write when a bounded wait gives up and never read."""
    if torch.cuda.is_current_stream_capturing():
        raise RuntimeError("make one call outside of the graph first: it allocates the device's status word")
    ws = torch.zeros(L.TILEQ_GROUPED_WS_BYTES, dtype=torch.uint8, device=torch.device("cuda", index))
    torch.cuda.current_stream(index).synchronize()  # zeroed before a call on any other stream
    return _status_words.setdefault(index, (ws, ws.data_ptr()))  # of two threads' words the first stays


def expert_status(device="cuda") -> int:
    """Synchronously read and clear the first device error of these calls (0: none), as tileq_device_status."""
    device = torch.device(device)
    index = torch.cuda.current_device() if device.index is None else device.index
    with torch.cuda.device(index):
        torch.cuda.synchronize()
        return L.tileq_device_status((_status_words.get(index) or _status_word(index))[0])


def _elsewhere(index: int, stream, call, *tensors):
    """call() with device `index` and the given stream (or the device's own) current: where a call is not for the
    current device's current stream.  New outputs belong to the stream they are made on; the memory of the given
    tensors is not handed out again before that stream has come past the call."""
    if stream is None:
        stream = torch.cuda.current_stream(index)
    elif isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device=torch.device("cuda", index))
    if stream.device.index != index:
        raise ValueError(f"the stream is on {stream.device}, the tensors are on cuda:{index}")
    with torch.cuda.stream(stream):
        result = call()
    for t in tensors:
        if t is not None:
            t.record_stream(stream)
    return result


def _check(status: int, name: str):
    if status:
        raise L.TileQError(status, name)


def _unrecorded():
    """An operand requires a gradient: no gradient may be lost silently, so refuse what autograd would have to record."""
    if torch.is_grad_enabled():
        raise ValueError("autograd does not record this product, and an operand requires a gradient: call it under "
                         "torch.no_grad() or in a torch.autograd.Function")


def _rows(t: torch.Tensor, name: str, index: int):
    """(rows, columns, row stride) of a matrix on device `index`; the stride of a single row is 0, contiguous."""
    if t.get_device() != index or index < 0:
        raise ValueError(f"{name} is on {t.device}: all tensors must be on the same GPU")
    shape, stride = t.shape, t.stride()
    if len(shape) != 2:
        raise ValueError(f"{name} must be a matrix, not of shape {tuple(shape)}")
    n, c = shape
    if c < 1:
        raise ValueError(f"{name} has no columns")
    if n <= 1:
        if n and stride[1] != 1 and c > 1:
            raise ValueError(f"{name} must be contiguous in its last dimension")
        return n, c, 0
    if (stride[1] != 1 and c > 1) or stride[0] < c:
        raise ValueError(f"{name} must be contiguous in its last dimension, with rows that do not overlap")
    return n, c, stride[0]


def _weights(t: torch.Tensor, name: str, index: int):
    """(E, d_out, d_in, row stride, expert stride) of weights [E, d_out, d_in] on device `index`."""
    if t.get_device() != index or index < 0:
        raise ValueError(f"{name} is on {t.device}: all tensors must be on the same GPU")
    shape, stride = t.shape, t.stride()
    if len(shape) != 3:
        raise ValueError(f"{name} must be [E, d_out, d_in], not of shape {tuple(shape)}")
    E, O, I = shape
    if not 1 <= E <= L.TILEQ_GROUPED_MAX_E or O < 1 or I < 1:
        raise ValueError(f"{name}: 1 to {L.TILEQ_GROUPED_MAX_E} experts and no empty widths, not {tuple(shape)}")
    ld = stride[1] if O > 1 else I
    if (stride[2] != 1 and I > 1) or ld < I or (E > 1 and stride[0] < (O - 1) * ld + I):
        raise ValueError(f"{name} must be contiguous in its last dimension, with rows that do not overlap")
    return E, O, I, ld, (stride[0] if E > 1 else 0)


def _vector(t, n: int, dtype, name: str, index: int) -> int:
    """Pointer of a contiguous vector of n values, 0 for none."""
    if t is None:
        return 0
    if t.dtype is not dtype or t.get_device() != index or t.dim() != 1 or t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of {n} values on cuda:{index}")
    return t.data_ptr()


def _no_offsets(E: int) -> int:
    """None for the offsets: one expert has every row."""
    if E != 1:
        raise ValueError(f"{E} experts need expert_offsets")
    return 0


def _result(out, out_dtype, default, shape, like: torch.Tensor) -> torch.Tensor:
    """The given result, checked, or a new one."""
    if out is None:
        if out_dtype is None:
            out_dtype = default
        if out_dtype not in _CODE:
            raise ValueError("out_dtype must be bfloat16, float16 or float32")
        return like.new_empty(shape) if out_dtype is like.dtype else like.new_empty(shape, dtype=out_dtype)
    if out.dtype not in _CODE or (out_dtype is not None and out.dtype is not out_dtype):
        raise ValueError("out must be bfloat16, float16 or float32, as out_dtype says")
    if out.shape != shape:
        raise ValueError(f"out must be of shape {tuple(shape)}")
    return out


def _operands(a: torch.Tensor, b: torch.Tensor) -> int:
    """The type code of two 16-bit operands."""
    dtype = a.dtype
    code = _OPERAND.get(dtype)
    if code is None or b.dtype is not dtype:
        raise ValueError(f"the operands must both be bfloat16 or both float16, not {dtype} and {b.dtype}")
    return code


def grouped_gemm(x, w, expert_offsets, out=None, out_dtype=None, stream=None):
    """y [P, d_out] with y[p] = W_e x[p]: x [P, d_in], w [E, d_out, d_in]."""
    if x.requires_grad or w.requires_grad or (out is not None and out.requires_grad):
        _unrecorded()
    code, index = _operands(x, w), x.get_device()
    P, I, ld_x = _rows(x, "x", index)
    E, O, Iw, ld_w, stride_w = _weights(w, "w", index)
    if I != Iw:
        raise ValueError(f"x has {I} columns, w expects {Iw}")
    off = _no_offsets(E) if expert_offsets is None else _vector(expert_offsets, E + 1, _I32, "expert_offsets", index)
    if stream is not None or torch.cuda.current_device() != index:
        return _elsewhere(index, stream, lambda: grouped_gemm(x, w, expert_offsets, out, out_dtype),
                          x, w, expert_offsets, out)
    y = _result(out, out_dtype, x.dtype, (P, O), x)
    ld_y = 0 if out is None else _rows(y, "out", index)[2]
    g = L.tileq_grouped(code, _CODE[y.dtype], E, P, I, O, ld_x, ld_y, ld_w, stride_w, off)
    word = _status_words.get(index) or _status_word(index)
    _check(L.lib().tileq_grouped_gemm(byref(g), x.data_ptr(), w.data_ptr(), y.data_ptr(), word[1], L.TILEQ_GROUPED_WS_BYTES,
                                      torch._C._cuda_getCurrentRawStream(index)), "tileq_grouped_gemm")
    if out is not None:
        _written(out)
    return y


def grouped_gemm_dx(dy, w, expert_offsets, out=None, out_dtype=None, stream=None):
    """dx [P, d_in] with dx[p] = W_e^T dy[p]: dy [P, d_out], w [E, d_out, d_in]."""
    if dy.requires_grad or w.requires_grad or (out is not None and out.requires_grad):
        _unrecorded()
    code, index = _operands(dy, w), dy.get_device()
    P, O, ld_y = _rows(dy, "dy", index)
    E, Ow, I, ld_w, stride_w = _weights(w, "w", index)
    if O != Ow:
        raise ValueError(f"dy has {O} columns, w expects {Ow}")
    off = _no_offsets(E) if expert_offsets is None else _vector(expert_offsets, E + 1, _I32, "expert_offsets", index)
    if stream is not None or torch.cuda.current_device() != index:
        return _elsewhere(index, stream, lambda: grouped_gemm_dx(dy, w, expert_offsets, out, out_dtype),
                          dy, w, expert_offsets, out)
    dx = _result(out, out_dtype, dy.dtype, (P, I), dy)
    ld_x = 0 if out is None else _rows(dx, "out", index)[2]
    g = L.tileq_grouped(code, _CODE[dx.dtype], E, P, I, O, ld_x, ld_y, ld_w, stride_w, off)
    word = _status_words.get(index) or _status_word(index)
    _check(L.lib().tileq_grouped_gemm_dx(byref(g), dy.data_ptr(), w.data_ptr(), dx.data_ptr(), word[1],
                                         L.TILEQ_GROUPED_WS_BYTES, torch._C._cuda_getCurrentRawStream(index)),
           "tileq_grouped_gemm_dx")
    if out is not None:
        _written(out)
    return dx


def grouped_gemm_dw(x, dy, expert_offsets, out=None, out_dtype=None, stream=None):
    """dW [E, d_out, d_in] with dW_e = sum over the rows p of e of dy[p] x[p]^T, zeros for an expert without rows."""
    if x.requires_grad or dy.requires_grad or (out is not None and out.requires_grad):
        _unrecorded()
    code, index = _operands(x, dy), x.get_device()
    P, I, ld_x = _rows(x, "x", index)
    Py, O, ld_y = _rows(dy, "dy", index)
    if P != Py:
        raise ValueError(f"x has {P} rows, dy {Py}")
    E = 1 if expert_offsets is None else expert_offsets.numel() - 1
    if not 1 <= E <= L.TILEQ_GROUPED_MAX_E:
        raise ValueError(f"expert_offsets must hold 2 to {L.TILEQ_GROUPED_MAX_E + 1} values")
    off = _no_offsets(E) if expert_offsets is None else _vector(expert_offsets, E + 1, _I32, "expert_offsets", index)
    if stream is not None or torch.cuda.current_device() != index:
        return _elsewhere(index, stream, lambda: grouped_gemm_dw(x, dy, expert_offsets, out, out_dtype),
                          x, dy, expert_offsets, out)
    dw = _result(out, out_dtype, x.dtype, (E, O, I), x)
    ld_w, stride_w = (0, 0) if out is None else _weights(dw, "out", index)[3:]
    g = L.tileq_grouped(code, _CODE[dw.dtype], E, P, I, O, ld_x, ld_y, ld_w, stride_w, off)
    word = _status_words.get(index) or _status_word(index)
    _check(L.lib().tileq_grouped_gemm_dw(byref(g), x.data_ptr(), dy.data_ptr(), dw.data_ptr(), word[1],
                                         L.TILEQ_GROUPED_WS_BYTES, torch._C._cuda_getCurrentRawStream(index)),
           "tileq_grouped_gemm_dw")
    if out is not None:
        _written(out)
    return dw


# ------------------------------------------------------------------ fp8
def _quantised(q, shape, like: torch.Tensor) -> torch.Tensor:
    """The given e4m3 tensor, checked, or a new one whose rows start at multiples of 16 bytes, as the product reads them."""
    if q is None:
        width = shape[-1]
        if width % 16 == 0:
            return like.new_empty(shape, dtype=_F8)
        return like.new_empty((*shape[:-1], -(-width // 16) * 16), dtype=_F8)[..., :width]
    if q.dtype is not _F8 or q.shape != shape:
        raise ValueError(f"out must be float8_e4m3fn of shape {tuple(shape)}")
    return q


def _scales(s, shape, index: int, name: str) -> int:
    """Row stride of a given scale tensor (0 where it has one row)."""
    if s.dtype is not _F32 or s.get_device() != index or s.shape != shape:
        raise ValueError(f"{name} must be float32 of shape {tuple(shape)} on cuda:{index}")
    if len(shape) > 2:
        if not s.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        return 0
    stride = s.stride()
    if (stride[1] != 1 and shape[1] > 1) or (shape[0] > 1 and stride[0] < shape[1]):
        raise ValueError(f"{name} must be contiguous in its last dimension, with rows that do not overlap")
    return stride[0] if shape[0] > 1 else 0


def fp8_quantize(x, rows=None, swiglu=False, row_scale=None, out=None, scales=None, stream=None):
    """Rows in e4m3 with a scale for every 128 columns: (q [R, C], scales [ceil(C / 128), R]).

    x [T, C] (swiglu: [T, 2C], gate then up, of which silu(gate) * up is quantised) in bf16, fp16
    or fp32, C up to 65535 * 1024.  rows: int32 [R], the row of x of each row of q (outside [0, T): zeros); without it
    R = T.  row_scale: fp32 [R], a factor of each row of q.
    """
    code = _CODE.get(x.dtype)
    if code is None:
        raise ValueError("x must be bfloat16, float16 or float32")
    index = x.get_device()
    T, C, ld_x = _rows(x, "x", index)
    if swiglu:
        if C % 2:
            raise ValueError("x must hold the gate's and the up projection's columns")
        C //= 2
    R = T if rows is None else rows.numel()
    at = _vector(rows, R, _I32, "rows", index)
    factor = _vector(row_scale, R, _F32, "row_scale", index)
    if stream is not None or torch.cuda.current_device() != index:
        return _elsewhere(index, stream, lambda: fp8_quantize(x, rows, swiglu, row_scale, out, scales),
                          x, rows, row_scale, out, scales)
    q, shape = _quantised(out, (R, C), x), (-(-C // 128), R)
    if scales is None:
        s, ld_s = x.new_empty(shape, dtype=_F32), 0
    else:
        s, ld_s = scales, _scales(scales, shape, index, "scales")
    a = L.tileq_fp8_rows(code, R, T, C, 1 if swiglu else 0, at, factor, ld_x, _rows(q, "out", index)[2], ld_s)
    _check(L.lib().tileq_fp8_quantize(byref(a), x.data_ptr(), q.data_ptr(), s.data_ptr(),
                                      torch._C._cuda_getCurrentRawStream(index)), "tileq_fp8_quantize")
    if out is not None:
        _written(out)
    if scales is not None:
        _written(scales)
    return q, s


def fp8_quantize_weights(w, out=None, scales=None, stream=None):
    """Weights [E, d_out, d_in] (or one expert's [d_out, d_in]) in e4m3 with a scale for every 128 x 128 block:
    (q like w, scales [E, ceil(d_out / 128), ceil(d_in / 128)], without E for one)."""
    code = _CODE.get(w.dtype)
    if code is None:
        raise ValueError("w must be bfloat16, float16 or float32")
    if w.dim() == 2:
        q, s = fp8_quantize_weights(w[None], None if out is None else out[None], None if scales is None else scales[None],
                                    stream)
        return q[0], s[0]
    index = w.get_device()
    E, O, I, ld_w, stride_w = _weights(w, "w", index)
    if stream is not None or torch.cuda.current_device() != index:
        return _elsewhere(index, stream, lambda: fp8_quantize_weights(w, out, scales), w, out, scales)
    q, shape = _quantised(out, (E, O, I), w), (E, -(-O // 128), -(-I // 128))
    ld_q, stride_q = _weights(q, "out", index)[3:]
    if scales is None:
        s = w.new_empty(shape, dtype=_F32)
    else:
        s = scales
        _scales(s, shape, index, "scales")
    g = L.tileq_grouped(code, 0, E, 0, I, O, 0, 0, ld_w, stride_w, 0)
    _check(L.lib().tileq_fp8_quantize_weights(byref(g), w.data_ptr(), q.data_ptr(), ld_q, stride_q, s.data_ptr(),
                                              torch._C._cuda_getCurrentRawStream(index)), "tileq_fp8_quantize_weights")
    if out is not None:
        _written(out)
    if scales is not None:
        _written(scales)
    return q, s


def fp8_gemm(xq, xs, wq, ws, expert_offsets=None, out=None, out_dtype=None, stream=None):
    """y [P, d_out] (bf16, or out_dtype) from e4m3 rows xq [P, d_in] with scales xs [ceil(d_in / 128), P]
    and e4m3 weights wq [E, d_out, d_in] with scales ws [E, ceil(d_out / 128), ceil(d_in / 128)].

    Dense, without expert_offsets: wq [d_out, d_in], ws [ceil(d_out / 128), ceil(d_in / 128)].
    """
    if xs.requires_grad or ws.requires_grad or (out is not None and out.requires_grad):
        _unrecorded()
    if (wq.dim() == 2) != (expert_offsets is None):
        raise ValueError("a product by expert takes wq [E, d_out, d_in] and expert_offsets, a dense one wq [d_out, d_in]")
    if xq.dtype is not _F8 or wq.dtype is not _F8:
        raise ValueError("xq and wq must be float8_e4m3fn")
    index = xq.get_device()
    P, I, ld_x = _rows(xq, "xq", index)
    kb = -(-I // 128)
    if expert_offsets is None:
        O, Iw, ld_w = _rows(wq, "wq", index)
        if O < 1:
            raise ValueError("wq has no rows")
        E, stride_w, blocks = 1, 0, (-(-O // 128), kb)
    else:
        E, O, Iw, ld_w, stride_w = _weights(wq, "wq", index)
        blocks = (E, -(-O // 128), kb)
    if I != Iw:
        raise ValueError(f"xq has {I} columns, wq expects {Iw}")
    ld_xs = _scales(xs, (kb, P), index, "xs")
    if not ws.is_contiguous():
        raise ValueError("ws must be contiguous")
    _scales(ws, blocks, index, "ws")
    off = _vector(expert_offsets, E + 1, _I32, "expert_offsets", index)
    if stream is not None or torch.cuda.current_device() != index:
        return _elsewhere(index, stream, lambda: fp8_gemm(xq, xs, wq, ws, expert_offsets, out, out_dtype),
                          xq, xs, wq, ws, expert_offsets, out)
    y = _result(out, out_dtype, torch.bfloat16, (P, O), xq)
    ld_y = 0 if out is None else _rows(y, "out", index)[2]
    g = L.tileq_grouped(L.TILEQ_DT_E4M3, _CODE[y.dtype], E, P, I, O, ld_x, ld_y, ld_w, stride_w, off)
    word = _status_words.get(index) or _status_word(index)
    _check(L.lib().tileq_fp8_gemm(byref(g), xq.data_ptr(), xs.data_ptr(), ld_xs, wq.data_ptr(), ws.data_ptr(), y.data_ptr(),
                                  word[1], L.TILEQ_GROUPED_WS_BYTES, torch._C._cuda_getCurrentRawStream(index)),
           "tileq_fp8_gemm")
    if out is not None:
        _written(out)
    return y
