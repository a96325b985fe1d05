"""Cases of the experts' products: what they compute, in plain torch, and how long they take.

The operators of an uncompressed expert layer, beside the TileQ layer:

  fwd      y[p] = W_e x[p] for the rows p of expert e            (tq.grouped_gemm)
  dx       dx[p] = W_e^T dy[p]                                   (tq.grouped_gemm_dx)
  dw       dW_e = sum over the rows p of e of dy[p] x[p]^T       (tq.grouped_gemm_dw)
  quant    rows of x in e4m3, one power-of-two scale per 128     (tq.fp8_quantize)
  quantw   weights in e4m3, one scale per 128 x 128 block        (tq.fp8_quantize_weights)
  fp8      y[p] = W_e x[p] from such rows and weights            (tq.fp8_gemm)
  down     SwiGLU and its quantisation, then the fp8 product     (tq.fp8_quantize, tq.fp8_gemm)

Rows are sorted by expert; expert e holds rows expert_offsets[e] .. expert_offsets[e + 1] - 1, as the
routing of the layer leaves them.  `own` picks the framework's calls; otherwise the plain form runs.
"""
import math

import numpy as np
import torch

own = False

E4M3_MAX = 448.0


# ------------------------------------------------------------------ cases
def _case(op, E, T, k, d_in, d_out, dtype="bf16", sigma=1.0, zipf=0.0, **more):
    return dict(op=op, E=E, T=T, k=k, d_in=d_in, d_out=d_out, dtype=dtype, sigma=sigma, zipf=zipf, **more)


def listed():
    return [
        # the smallest layer of the seeded workloads, 64 tokens: a call's latency
        dict(_case("fwd", 4, 64, 2, 256, 512), name="fwd-tiny-4e-T64"),
        # one token through the gate projection of an 8-expert layer: two experts' weights, read once
        dict(_case("fwd", 8, 1, 2, 4096, 14336), name="fwd-8e-T1"),
        # a small serving batch on 60 skewed experts: ragged, about 17 rows an expert, some none, fp16
        dict(_case("fwd", 60, 256, 4, 2048, 1408, "fp16", zipf=1.1), name="fwd-60e-T256"),
        # the long prefill of the 64-expert layer: 131072 rows, the largest product
        dict(_case("fwd", 64, 16384, 8, 4096, 1536), name="fwd-64e-T16384"),
        # training, gradient of the activations of a 60-expert layer with a skewed load
        dict(_case("dx", 60, 2048, 4, 2048, 1408, zipf=1.1), name="dx-60e-T2048"),
        # training, gradient of the up projection of the 8-expert layer: 4.7e8 weights
        dict(_case("dw", 8, 4096, 2, 4096, 14336, sigma=1.5), name="dw-8e-T4096"),
        # odd sizes: a width that no tile divides, 333 tokens on seven experts, fp16
        dict(_case("dw", 7, 333, 2, 1000, 696, "fp16"), name="dw-odd-7e-T333"),
        # tokens gathered to their experts' rows and quantised, long prefill of the 64-expert layer
        dict(_case("quant", 64, 16384, 8, 4096, 0), name="quant-64e-T16384"),
        # the same of a small serving batch
        dict(_case("quant", 60, 16, 4, 2048, 0), name="quant-60e-T16"),
        # a decode batch of 16 tokens on 64 experts in fp8: two rows an expert, weights dominate
        dict(_case("fp8", 64, 16, 8, 4096, 1536), name="fp8-64e-T16"),
        # the always-on shared expert of the 60-expert layer, dense, in fp8
        dict(_case("fp8", 1, 2048, 1, 2048, 5632, dense=True), name="fp8-dense-T2048"),
        # SwiGLU, quantisation and the down projection of the 8-expert layer at prefill, in fp8
        dict(_case("down", 8, 4096, 2, 14336, 4096, sigma=1.5), name="down-8e-T4096"),
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """A case of the ranges that the listed ones stand for."""
    while True:
        op = rng.choice(["fwd", "dx", "dw", "fwd", "quant", "quantw", "fp8", "down"])
        E = _log_uniform(rng, 1, 64)
        k = rng.randint(1, min(8, E))
        T = _log_uniform(rng, 1, 16384)
        step = 16 if op in ("fp8", "down", "quant", "quantw") else 8
        d_in = step * _log_uniform(rng, 96 // step, 14336 // step)
        d_out = step * _log_uniform(rng, 96 // step, 14336 // step)
        dense = op == "fp8" and rng.random() < 0.25
        c = _case(op, 1 if dense else E, T, 1 if dense else k, d_in, 0 if op == "quant" else d_out,
                  rng.choice(["bf16", "bf16", "fp16"]), rng.choice([1.0, 1.5]), rng.choice([0.0, 1.1]))
        if dense:
            c["dense"] = True
        # no dearer than the largest listed case in any of work, weights and rows
        w = work(c)
        rows = T * k * (d_in * (2 if op == "down" else 1) + d_out)
        if w["flops"] <= 1.6e12 and E * d_in * max(d_out, 1) <= 4.7e8 and rows <= 7.3e8 and w["bytes"] <= 1.9e9:
            return c


def _route(case, seed):
    """Expert of each (token, choice) pair: the top k of the logits, with the load's skew."""
    T, E, k = case["T"], case["E"], case["k"]
    rng = np.random.default_rng([seed, T, E, k])
    logits = rng.standard_normal((T, E), dtype=np.float32) * np.float32(case["sigma"])
    if case["zipf"]:
        logits += (-case["zipf"] * np.log1p(rng.permutation(E))).astype(np.float32)
    return np.argsort(-logits, axis=1, kind="stable")[:, :k] if k < E else np.tile(np.arange(E), (T, 1))


def _counts(case, seed):
    return np.bincount(_route(case, seed).reshape(-1), minlength=case["E"])


def _dtype(case):
    return {"bf16": torch.bfloat16, "fp16": torch.float16}[case["dtype"]]


def _blocks(n):
    return -(-n // 128)


# ------------------------------------------------------------------ inputs
def _pow2_scale(amax):
    """The smallest power of two s with amax / s <= 448, at least 2^-126; 1 for a block of zeros."""
    m, e = torch.frexp(amax)  # amax = m 2^e, 1/2 <= m < 1;  448 = 7/8 * 2^9
    e = torch.clamp(e + (m > 0.875).to(e.dtype) - 9, min=-126)
    return torch.where(amax > 0, torch.ldexp(torch.ones_like(amax), e), torch.ones_like(amax))


def _pad128(x, dims):
    pad = [0, 0] * x.dim()
    for d in dims:
        pad[2 * (x.dim() - 1 - d) + 1] = -x.shape[d] % 128
    return torch.nn.functional.pad(x, pad)


def _quant_rows(x):
    """(e4m3 [R, C], fp32 scales [ceil(C / 128), R]) of fp32 rows."""
    R, C = x.shape
    b = _pad128(x, [1]).view(R, -1, 128)
    s = _pow2_scale(b.abs().amax(-1))
    q = (b / s[..., None]).to(torch.float8_e4m3fn).view(R, -1)[:, :C]
    return q.contiguous(), s.t().contiguous()


def _quant_weights(w):
    """(e4m3 [E, O, I], fp32 scales [E, ceil(O / 128), ceil(I / 128)]) of fp32 weights."""
    E, O, I = w.shape
    b = _pad128(w, [1, 2]).view(E, _blocks(O), 128, _blocks(I), 128)
    s = _pow2_scale(b.abs().amax((2, 4)))
    q = (b / s[:, :, None, :, None]).to(torch.float8_e4m3fn).view(E, _blocks(O) * 128, -1)[:, :O, :I]
    return q.contiguous(), s


def prepare(case, seed):
    E, T, k, d_in, d_out = case["E"], case["T"], case["k"], case["d_in"], case["d_out"]
    op, dt = case["op"], _dtype(case)
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, std=1.0, dtype=dt):
        return torch.randn(*shape, generator=g, device="cuda").mul_(std).to(dtype)

    def weights():
        w = torch.empty(E, d_out, d_in, dtype=dt, device="cuda")
        for e in range(E):
            w[e] = normal(d_out, d_in, std=d_in ** -0.5)
        return w

    experts = _route(case, seed).reshape(-1)
    counts = np.bincount(experts, minlength=E)
    offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    P = T * k
    s = {"op": op, "dtype": dt, "ends": [int(v) for v in offsets], "dense": bool(case.get("dense")),
         "offsets": torch.from_numpy(offsets).cuda()}
    if op in ("fwd", "dx"):
        s["w"] = weights()
        s["x"] = normal(P, d_in) if op == "fwd" else normal(P, d_out, std=0.02)
    elif op == "dw":
        s["x"], s["dy"] = normal(P, d_in), normal(P, d_out, std=0.02)
    elif op == "quant":
        s["x"] = normal(T, d_in)
        s["rows"] = torch.from_numpy((np.argsort(experts, kind="stable") // k).astype(np.int32)).cuda()
    elif op == "quantw":
        s["w"] = weights()
    else:
        s["wq"] = torch.empty(E, d_out, d_in, dtype=torch.float8_e4m3fn, device="cuda")
        s["ws"] = torch.empty(E, _blocks(d_out), _blocks(d_in), device="cuda")
        for e in range(E):
            q, sc = _quant_weights(normal(1, d_out, d_in, std=d_in ** -0.5, dtype=torch.float32))
            s["wq"][e], s["ws"][e] = q[0], sc[0]
        if op == "fp8":
            s["xq"], s["xs"] = _quant_rows(normal(P, d_in, dtype=torch.float32))
        else:
            s["x"] = normal(P, 2 * d_in)
            s["weight"] = torch.rand(P, generator=g, device="cuda")
    return s


# ------------------------------------------------------------------ one pass
def _plain(s):
    op, ends = s["op"], s["ends"]
    spans = list(zip(range(len(ends) - 1), ends[:-1], ends[1:]))
    if op == "fwd":
        return torch.cat([s["x"][a:b].float() @ s["w"][e].float().t() for e, a, b in spans if b > a]).to(s["dtype"])
    if op == "dx":
        return torch.cat([s["x"][a:b].float() @ s["w"][e].float() for e, a, b in spans if b > a]).to(s["dtype"])
    if op == "dw":
        return torch.stack([s["dy"][a:b].float().t() @ s["x"][a:b].float() for e, a, b in spans]).to(s["dtype"])
    if op == "quant":
        return _quant_rows(s["x"].float()[s["rows"].long()])
    if op == "quantw":
        return _quant_weights(s["w"].float())
    if op == "down":
        g, u = s["x"].float().chunk(2, dim=1)
        xq, xs = _quant_rows(g / (1 + torch.exp(-g)) * u * s["weight"][:, None])
    else:
        xq, xs = s["xq"], s["xs"]
    R, I = xq.shape
    x = xq.float() * xs.t().repeat_interleave(128, 1)[:, :I]
    O = s["wq"].shape[1]
    wide = [s["ws"][e].repeat_interleave(128, 0)[:O].repeat_interleave(128, 1)[:, :I] for e, a, b in spans if b > a]
    live = [(e, a, b) for e, a, b in spans if b > a]
    return torch.cat([x[a:b] @ (s["wq"][e].float() * sc).t() for (e, a, b), sc in zip(live, wide)]).to(torch.bfloat16)


def run(state):
    s = state
    if not own:
        return _plain(s)
    import tiled_rank_b200 as tq
    op = s["op"]
    if op == "fwd":
        return tq.grouped_gemm(s["x"], s["w"], s["offsets"])
    if op == "dx":
        return tq.grouped_gemm_dx(s["x"], s["w"], s["offsets"])
    if op == "dw":
        return tq.grouped_gemm_dw(s["x"], s["dy"], s["offsets"])
    if op == "quant":
        return tq.fp8_quantize(s["x"], rows=s["rows"])
    if op == "quantw":
        return tq.fp8_quantize_weights(s["w"])
    if op == "down":
        xq, xs = tq.fp8_quantize(s["x"], swiglu=True, row_scale=s["weight"])
        return tq.fp8_gemm(xq, xs, s["wq"], s["ws"], s["offsets"])
    if s["dense"]:
        return tq.fp8_gemm(s["xq"], s["xs"], s["wq"][0], s["ws"][0])
    return tq.fp8_gemm(s["xq"], s["xs"], s["wq"], s["ws"], s["offsets"])


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    E, T, k, d_in, d_out, op = (case[n] for n in ("E", "T", "k", "d_in", "d_out", "op"))
    P, w = T * k, d_in * d_out
    if op == "quant":  # x once, the row numbers, the e4m3 rows and their scales
        return {"bytes": 2 * T * d_in + 4 * P + P * d_in + 4 * P * _blocks(d_in), "flops": 2 * P * d_in}
    if op == "quantw":
        return {"bytes": 3 * E * w + 4 * E * _blocks(d_in) * _blocks(d_out), "flops": 2 * E * w}
    live = int((_counts(case, 0) > 0).sum())  # experts without rows are not read
    flops = 2 * P * w
    if op == "dw":
        return {"bytes": 2 * P * (d_in + d_out) + 2 * E * w, "flops": flops}
    if op in ("fwd", "dx"):
        return {"bytes": 2 * P * (d_in + d_out) + 2 * live * w, "flops": flops}
    ws = live * (w + 4 * _blocks(d_in) * _blocks(d_out))
    if op == "down":
        return {"bytes": 2 * P * (2 * d_in + d_out) + 4 * P + ws, "flops": flops}
    return {"bytes": P * (d_in + 4 * _blocks(d_in) + 2 * d_out) + ws, "flops": flops}


# ------------------------------------------------------------------ the definition, in 64 bits
def _e4m3(v):
    """v rounded to e4m3 (nearest, ties to even), |v| <= 448: steps of 2^(e - 3), at least 2^-9."""
    _, e = torch.frexp(v)  # |v| in [2^(e - 1), 2^e)
    step = torch.ldexp(torch.ones_like(v), torch.clamp(e - 4, min=-9))
    return torch.round(v / step) * step


def _exact_quant(x, rows):
    """Values and scales of blocks of `rows` x 128 of x [..., R, C] in 64 bits."""
    R, C = x.shape[-2:]
    val, scales = torch.empty_like(x), x.new_empty(*x.shape[:-2], -(-R // rows), _blocks(C))
    for j in range(_blocks(C)):
        part = x[..., 128 * j:128 * (j + 1)]
        top = part.abs().amax(-1)
        if rows > 1:
            top = torch.nn.functional.pad(top, (0, -R % rows)).unflatten(-1, (-1, rows)).amax(-1)
        e = torch.clamp(torch.ceil(torch.log2(top / E4M3_MAX)), min=-126)
        s = torch.exp2(e)
        s = torch.where(top / s > E4M3_MAX, 2 * s, torch.where(top / (s / 2) <= E4M3_MAX, s / 2, s))  # log2's last place
        s = torch.where(top > 0, torch.clamp(s, min=2.0 ** -126), torch.ones_like(s))
        scales[..., j] = s
        val[..., 128 * j:128 * (j + 1)] = _e4m3(part / s.repeat_interleave(rows, -1)[..., :R, None])
    return val, scales


def exact(case, seed):
    s = prepare(case, seed)
    op, ends, E = s["op"], s["ends"], case["E"]
    d_in, d_out, P = case["d_in"], case["d_out"], case["T"] * case["k"]
    if op == "quant":
        val, sc = _exact_quant(s["x"].double(), 1)
        at = s["rows"].long()
        return val.float()[at], sc[at].t()
    if op == "quantw":
        val, sc = _exact_quant(s["w"].double(), 128)
        return val, sc
    if op == "dw":
        out = torch.zeros(E, d_out, d_in, dtype=torch.float64, device="cuda")
        for e in range(E):
            at = slice(ends[e], ends[e + 1])
            out[e] = torch.einsum("po,pi->oi", s["dy"][at].double(), s["x"][at].double())
        return out
    out = torch.empty(P, d_in if op == "dx" else d_out, dtype=torch.float64, device="cuda")
    if op in ("fwd", "dx"):
        for e in range(E):
            at = slice(ends[e], ends[e + 1])
            out[at] = torch.einsum("pi,oi->po" if op == "fwd" else "po,oi->pi", s["x"][at].double(), s["w"][e].double())
        return out
    for e in range(E):
        at = slice(ends[e], ends[e + 1])
        if ends[e] == ends[e + 1]:
            continue
        if op == "down":
            both = s["x"][at].double()
            h = both[:, :d_in] * torch.sigmoid(both[:, :d_in]) * both[:, d_in:] * s["weight"][at, None].double()
            val, sc = _exact_quant(h, 1)
        else:
            val, sc = s["xq"][at].float().double(), s["xs"].t()[at].double()
        acc = torch.zeros(ends[e + 1] - ends[e], d_out, dtype=torch.float64, device="cuda")
        wscale = s["ws"][e].double()
        for j in range(_blocks(d_in)):
            cols = slice(128 * j, min(d_in, 128 * (j + 1)))
            part = val[:, cols] @ s["wq"][e][:, cols].float().double().t()
            acc += part * sc[:, j, None] * wscale[:, j].repeat_interleave(128)[None, :d_out]
        out[at] = acc
    return out
