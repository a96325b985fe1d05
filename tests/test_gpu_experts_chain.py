"""The experts' products together, as a layer uses them: routing, gather, gate and up, SwiGLU, down, combine;
in fp8 for serving, and in bf16 with the backward pass for training."""
import pytest

from experts_util import (assert_within, dequant_rows, dequant_weights, fp8_terms, ref_forward, ref_quant_rows)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tq():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import tiled_rank_b200 as tq
    yield tq
    assert tq.expert_status() == 0


def _routed(tq, T, E, k, seed):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    dev = "cuda"
    route = {"topk_idx": torch.empty(T, k, dtype=torch.int32, device=dev), "topk_w": torch.empty(T, k, device=dev),
             "expert_offsets": torch.empty(E + 1, dtype=torch.int32, device=dev),
             "sorted_pairs": torch.empty(T * k, dtype=torch.int32, device=dev)}
    ws = torch.zeros(64 << 20, dtype=torch.uint8, device=dev)
    tq.tileq_route(torch.randn(T, E, generator=g, device=dev) * 1.5, T, E, k, route, ws)
    pairs = route["sorted_pairs"]
    return g, route["expert_offsets"], (pairs // k).to(torch.int32), route["topk_w"].view(-1)[pairs.long()], pairs.long()


@pytest.mark.parametrize("T,E,k,D,F", [(1, 8, 2, 256, 512), (16, 60, 4, 512, 176), (700, 8, 2, 384, 320),
                                       (1024, 64, 8, 256, 192)])
def test_fp8_layer(tq, T, E, k, D, F):
    """Each product and quantisation of the layer against 64 bits on its own inputs, then the whole chain's output
    once more in a captured graph, bit by bit."""
    import torch
    g, off, rows, weight, pairs = _routed(tq, T, E, k, T)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x = rnd(T, D).to(torch.bfloat16)
    w1, s1 = tq.fp8_quantize_weights((rnd(E, 2 * F, D) * D ** -0.5).to(torch.bfloat16))
    w2, s2 = tq.fp8_quantize_weights((rnd(E, D, F) * F ** -0.5).to(torch.bfloat16))
    y = torch.empty(T * k, D, dtype=torch.float32, device="cuda")

    def layer():
        xq, xs = tq.fp8_quantize(x, rows=rows)
        gu = tq.fp8_gemm(xq, xs, w1, s1, off)
        hq, hs = tq.fp8_quantize(gu, swiglu=True, row_scale=weight)
        tq.fp8_gemm(hq, hs, w2, s2, off, out=y)
        return xq, xs, gu, hq, hs, torch.zeros(T * k, D, device="cuda").index_copy_(0, pairs, y).view(T, k, D).sum(1)

    xq, xs, gu, hq, hs, out = layer()
    rq, rs = ref_quant_rows(x.double()[rows.long()])
    assert torch.equal(xq.float().double(), rq) and torch.equal(xs.double(), rs)
    ref, mag = ref_forward(dequant_rows(xq, xs), dequant_weights(w1, s1), off)
    assert_within(gu, ref, mag, fp8_terms(D), "gate and up")
    h = gu.double()
    h = h[:, :F] * torch.sigmoid(h[:, :F]) * h[:, F:] * weight.double()[:, None]
    sc = hs.t().double().repeat_interleave(128, 1)[:, :F]
    assert ((dequant_rows(hq, hs) - h).abs() <= h.abs() * (2.0 ** -4 + 2.0 ** -20) + 2.0 ** -10 * sc).all()
    ref, mag = ref_forward(dequant_rows(hq, hs), dequant_weights(w2, s2), off)
    assert_within(y, ref, mag, fp8_terms(F), "down")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        again = layer()[-1]
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(again, out)


@pytest.mark.parametrize("T,E,k,D,F", [(40, 6, 2, 128, 256), (700, 8, 2, 384, 320)])
def test_training_step(tq, T, E, k, D, F):
    """Loss and gradients of a SwiGLU expert layer whose products are these calls, against autograd in 64 bits.

    Every value handed on in bf16 is rounded once, by 2^-8 of itself at most; from x to a weight's gradient there are
    up to six in a row (h, y's gradient, da or db, the gradient itself, each once or twice on the way), so the
    gradients' relative error in norm stays under 6 * 2^-8."""
    import torch
    g, off, rows, weight, pairs = _routed(tq, T, E, k, 3 * T)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    x, wg, wu, wd = rnd(T, D), rnd(E, F, D) / D ** 0.5, rnd(E, F, D) / D ** 0.5, rnd(E, D, F) / F ** 0.5
    target = rnd(T, D)
    at = rows.long()

    def backward():
        xp = x[at]
        a, b = tq.grouped_gemm(xp, wg, off, out_dtype=torch.float32), tq.grouped_gemm(xp, wu, off, out_dtype=torch.float32)
        sig = torch.sigmoid(a)
        h = (a * sig * b * weight[:, None]).to(torch.bfloat16)
        y = tq.grouped_gemm(h, wd, off, out_dtype=torch.float32)
        out = torch.zeros(T, D, device="cuda").index_add_(0, at, y)
        dy = (2 * (out - target.float()))[at].to(torch.bfloat16)
        dwd = tq.grouped_gemm_dw(h, dy, off)
        dh = tq.grouped_gemm_dx(dy, wd, off, out_dtype=torch.float32) * weight[:, None]
        da = (dh * b * (sig + a * sig * (1 - sig))).to(torch.bfloat16)
        db = (dh * a * sig).to(torch.bfloat16)
        dwg, dwu = tq.grouped_gemm_dw(xp, da, off), tq.grouped_gemm_dw(xp, db, off)
        dxp = tq.grouped_gemm_dx(da, wg, off, out_dtype=torch.float32) + tq.grouped_gemm_dx(db, wu, off, out_dtype=torch.float32)
        return dwg, dwu, dwd, torch.zeros(T, D, device="cuda").index_add_(0, at, dxp)

    got = backward()
    leaves = [t.double().requires_grad_() for t in (wg, wu, wd, x)]
    ends = off.tolist()
    Wg, Wu, Wd, X = leaves
    out = torch.zeros(T, D, dtype=torch.float64, device="cuda")
    for e in range(E):
        r = at[ends[e]:ends[e + 1]]
        hid = torch.nn.functional.silu(X[r] @ Wg[e].t()) * (X[r] @ Wu[e].t()) * weight[ends[e]:ends[e + 1], None].double()
        out = out.index_add(0, r, hid @ Wd[e].t())
    ((out - target.double()) ** 2).sum().backward()
    for name, v, leaf in zip(("gate", "up", "down", "x"), got, leaves):
        rel = ((v.double() - leaf.grad).norm() / leaf.grad.norm()).item()
        assert rel <= 6 * 2.0 ** -8, (name, rel)


def test_products_in_an_autograd_function(tq):
    """The way to train through the products: refused in a recorded place, right in a Function, for a leaf that is used
    twice.  The loss is the sum of y times a constant c that bf16 holds, so dy = c exactly and each gradient is one
    product: a leaf's is within the product's bound, and of two uses within that of the sum rounded once more."""
    import torch
    from experts_util import bound, offsets_of, ref_dw, ref_dx
    g = torch.Generator(device="cuda").manual_seed(11)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    counts, I, O = [20, 0, 130, 50], 136, 72
    off = offsets_of(counts, 0, "cuda")
    x, w, c = rnd(sum(counts), I).requires_grad_(), rnd(4, O, I).requires_grad_(), rnd(sum(counts), O)

    class Product(torch.autograd.Function):
        @staticmethod
        def forward(ctx, a, b):
            ctx.save_for_backward(a, b)
            return tq.grouped_gemm(a, b, off)

        @staticmethod
        def backward(ctx, dy):
            a, b = ctx.saved_tensors
            return tq.grouped_gemm_dx(dy, b, off), tq.grouped_gemm_dw(a, dy, off)

    with pytest.raises(ValueError, match="requires a gradient"):
        tq.grouped_gemm(x, w, off)
    with torch.no_grad():
        want = tq.grouped_gemm(x, w, off)
    assert torch.equal(Product.apply(x, w), want)
    for uses in (1, 2):
        x.grad = w.grad = None
        sum((Product.apply(x, w) * c).float().sum() for _ in range(uses)).backward()
        for leaf, (ref, mag), terms in ((x, ref_dx(c, w.detach(), off), O), (w, ref_dw(x.detach(), c, off), max(counts))):
            lim = uses * bound(leaf.dtype, ref, mag, terms)
            lim = lim + (uses > 1) * (uses * ref.abs() + lim) * torch.finfo(leaf.dtype).eps / 2
            assert ((leaf.grad.double() - uses * ref).abs() <= lim).all(), uses


def test_bindings_of_the_library(tq):
    """The calls as the C interface has them, structs filled by hand: the same results as on tensors."""
    import torch
    E, P, I, O = 3, 50, 160, 272
    g = torch.Generator(device="cuda").manual_seed(5)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()
    x, dy, w = rnd(P, I), rnd(P, O), rnd(E, O, I)
    off = torch.tensor([0, 7, 7, P], dtype=torch.int32, device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    call = tq.tileq_grouped(tq.TILEQ_DT_BF16, tq.TILEQ_DT_F32, E, P, I, O, 0, 0, 0, 0, off.data_ptr())
    y, dx, dw = (torch.empty(*s, device="cuda") for s in ((P, O), (P, I), (E, O, I)))
    tq.tileq_grouped_gemm(call, x, w, y, ws)
    tq.tileq_grouped_gemm_dx(call, dy, w, dx, ws)
    tq.tileq_grouped_gemm_dw(call, x, dy, dw, ws)
    f32 = torch.float32
    assert torch.equal(y, tq.grouped_gemm(x, w, off, out_dtype=f32))
    assert torch.equal(dx, tq.grouped_gemm_dx(dy, w, off, out_dtype=f32))
    assert torch.equal(dw, tq.grouped_gemm_dw(x, dy, off, out_dtype=f32))

    f8 = torch.float8_e4m3fn
    xq, xs = torch.empty(P, I, dtype=f8, device="cuda"), torch.empty(2, P, device="cuda")
    wq, sw = torch.empty(E, O, I, dtype=f8, device="cuda"), torch.empty(E, 3, 2, device="cuda")
    tq.tileq_fp8_quantize(tq.tileq_fp8_rows(tq.TILEQ_DT_BF16, P, P, I, 0, None, None, 0, 0, 0), x, xq, xs)
    tq.tileq_fp8_quantize_weights(call, w, wq, 0, 0, sw)
    call.dtype = tq.TILEQ_DT_E4M3
    y8 = torch.empty(P, O, device="cuda")
    tq.tileq_fp8_gemm(call, xq, xs, 0, wq, sw, y8, ws)
    want = [*tq.fp8_quantize(x), *tq.fp8_quantize_weights(w)]
    for a, b in zip((xq, xs, wq, sw), want):
        assert torch.equal(a.float(), b.float())
    assert torch.equal(y8, tq.fp8_gemm(*want, off, out_dtype=f32))
    assert tq.tileq_device_status(ws) == 0
