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
