"""Helpers of the tests of the experts' products: the definitions in 64 bits and their error bounds."""
from __future__ import annotations

import torch


def offsets_of(counts, first=0, device="cpu"):
    off = [first]
    for c in counts:
        off.append(off[-1] + c)
    return torch.tensor(off, dtype=torch.int32, device=device)


def bound(dtype, ref, mag, terms):
    """How far a sum of `terms` products, accumulated in fp32 and rounded once to `dtype`, may be from `ref`.

    ref is the sum in 64 bits, mag the sum of the products' magnitudes.  The products of two 8- or
    11-bit significands are exact in fp32.  Each addition errs by at most one unit (2^-23: the tensor
    core may cut rather than round) of a partial sum, which mag bounds: terms * 2^-23 * mag in all.
    The last rounding is off by half a step of `dtype` at the value, eps / 2 relative, or half the
    smallest step below the normal range.
    """
    fi = torch.finfo(dtype)
    acc = terms * 2.0 ** -23 * mag
    return acc + (ref.abs() + acc).clamp(min=fi.tiny) * (fi.eps / 2)


def assert_within(got, ref, mag, terms, what=""):
    err = (got.double() - ref).abs()
    lim = bound(got.dtype, ref, mag, terms)
    assert torch.isfinite(got).all(), f"{what}: non-finite"
    worst = (err / lim).max().item() if err.numel() else 0.0
    assert worst <= 1.0, f"{what}: {worst:.3g} times the bound"


def spans(off):
    off = off.tolist()
    return [(e, off[e], off[e + 1]) for e in range(len(off) - 1)]


def ref_forward(x, w, off):
    """(y, magnitudes) in 64 bits; rows of no expert are left zero."""
    y = torch.zeros(x.shape[0], w.shape[1], dtype=torch.float64, device=x.device)
    m = torch.zeros_like(y)
    for e, a, b in spans(off):
        xe, we = x[a:b].double(), w[e].double()
        y[a:b], m[a:b] = xe @ we.t(), xe.abs() @ we.abs().t()
    return y, m


def ref_dx(dy, w, off):
    d = torch.zeros(dy.shape[0], w.shape[2], dtype=torch.float64, device=dy.device)
    m = torch.zeros_like(d)
    for e, a, b in spans(off):
        ye, we = dy[a:b].double(), w[e].double()
        d[a:b], m[a:b] = ye @ we, ye.abs() @ we.abs()
    return d, m


def ref_dw(x, dy, off):
    E = off.shape[0] - 1
    d = torch.zeros(E, dy.shape[1], x.shape[1], dtype=torch.float64, device=x.device)
    m = torch.zeros_like(d)
    for e, a, b in spans(off):
        xe, ye = x[a:b].double(), dy[a:b].double()
        d[e], m[e] = ye.t() @ xe, ye.abs().t() @ xe.abs()
    return d, m


# ------------------------------------------------------------------ e4m3 with a scale per block of 128
def round_e4m3(v):
    """64-bit values of magnitude <= 448 rounded to e4m3, ties to even: steps 2^(exponent - 3), at least 2^-9."""
    _, e = torch.frexp(v)
    step = torch.ldexp(torch.ones_like(v), torch.clamp(e - 4, min=-9))
    return torch.round(v / step) * step


def block_scale(amax):
    """Smallest power of two s >= 2^-126 with amax / s <= 448 (1 for 0, NaN where amax is not finite), searched."""
    s = torch.full_like(amax, 2.0 ** -126)
    for _ in range(260):
        s = torch.where(amax / s > 448.0, s * 2, s)
    s = torch.where(amax == 0, torch.ones_like(s), s)
    return torch.where(torch.isfinite(amax), s, torch.full_like(s, float("nan")))


def ref_quant_rows(v):
    """(values / scale [R, C], scales [ceil(C / 128), R]) of 64-bit rows."""
    q, sc = torch.empty_like(v), []
    for c in range(0, v.shape[1], 128):
        part = v[:, c:c + 128]
        top = part.abs().amax(1)
        s = block_scale(torch.where(torch.isnan(part).any(1), torch.full_like(top, float("nan")), top))
        q[:, c:c + 128] = round_e4m3(part / s[:, None])
        sc.append(s)
    return q, torch.stack(sc)


def ref_quant_weights(w):
    E, O, I = w.shape
    q = torch.empty_like(w)
    s = torch.empty(E, -(-O // 128), -(-I // 128), dtype=torch.float64, device=w.device)
    for o in range(0, O, 128):
        for i in range(0, I, 128):
            part = w[:, o:o + 128, i:i + 128]
            s[:, o // 128, i // 128] = sc = block_scale(part.abs().amax((1, 2)))
            q[:, o:o + 128, i:i + 128] = round_e4m3(part / sc[:, None, None])
    return q, s


def dequant_rows(q, s):
    return q.float().double() * s.t().double().repeat_interleave(128, 1)[:, :q.shape[1]]


def dequant_weights(q, s):
    s = s.double().repeat_interleave(128, -2).repeat_interleave(128, -1)
    return q.float().double() * s[..., :q.shape[-2], :q.shape[-1]]


def fp8_terms(d_in):
    """Roundings of an fp8 product, in units of 2^-23 of the magnitudes: the additions of the products, and per
    block of 128 one rounding of the scales' product and one of the block's addition."""
    return d_in + 2 * -(-d_in // 128)
