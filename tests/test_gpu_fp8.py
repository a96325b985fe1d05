"""The fp8 products and their quantisers on the GPU against their definitions in 64 bits."""
import pytest

from experts_util import (assert_within, block_scale, dequant_rows, dequant_weights, fp8_terms, offsets_of,
                          ref_forward, ref_quant_rows, ref_quant_weights, round_e4m3)

pytestmark = pytest.mark.gpu

RAGGED = [0, 1, 15, 16, 17, 31, 32, 33, 0, 63, 64, 65, 127, 128, 129, 0]
LONG = [255, 256, 257, 0, 300, 513, 1, 700]
FEW = [0, 1, 0, 0, 2, 1, 0, 3]


@pytest.fixture(scope="module")
def tq():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import tiled_rank_b200 as tq
    yield tq
    assert tq.expert_status() == 0


def _rng(seed):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    return lambda *s: torch.randn(*s, generator=g, device="cuda")


def _same(got, want):
    """Equal values, NaN in the same places."""
    import torch
    got, want = got.float().double(), want.double()
    return torch.equal(got.isnan(), want.isnan()) and torch.equal(got.nan_to_num(), want.nan_to_num())


# ------------------------------------------------------------------ quantisers: exact
@pytest.mark.parametrize("dtype", ["bfloat16", "float16", "float32"])
@pytest.mark.parametrize("R,C", [(1, 1), (3, 128), (9, 129), (64, 2048), (17, 1000), (130, 1152), (5, 4104)])
def test_rows(tq, R, C, dtype):
    import torch
    x = (_rng(R * C)(R, C) * torch.logspace(-3, 3, R, device="cuda")[:, None]).to(getattr(torch, dtype))
    q, s = tq.fp8_quantize(x)
    rq, rs = ref_quant_rows(x.double())
    assert torch.equal(s.double(), rs) and _same(q, rq)


def test_every_16_bit_value_and_the_borders(tq):
    """All bf16 and fp16 values in blocks of their own magnitude, and maxima on both sides of every border."""
    import torch
    for dt in (torch.bfloat16, torch.float16):
        v = torch.arange(-32768, 32768, dtype=torch.int32, device="cuda").to(torch.int16).view(dt)
        v = v[torch.isfinite(v)]
        v = v[torch.argsort(v.abs().float())]
        v = torch.nn.functional.pad(v, (0, -v.numel() % 128)).view(-1, 128)
        q, s = tq.fp8_quantize(v)
        rq, rs = ref_quant_rows(v.double())
        assert torch.equal(s.double(), rs) and _same(q, rq)
    # fp32 maxima at 448 * 2^k and one unit to either side, with values on and next to e4m3's ties
    k = torch.arange(-140, 119, device="cuda", dtype=torch.float64)
    top = (448.0 * torch.exp2(k)).float()
    up, down = torch.nextafter(top, torch.full_like(top, float("inf"))), torch.nextafter(top, torch.zeros_like(top))
    for t in (top, up, down):
        tie = torch.tensor([17.0, 19.0, 8.5, 0.0078125 * 1.5, 2.0 ** -10, 3 * 2.0 ** -10, 2.0 ** -11, 240.0, 248.0],
                           device="cuda")
        x = t[:, None] * (tie / 448)
        x = torch.cat([t[:, None], x, torch.nextafter(x, torch.full_like(x, float("inf"))),
                       torch.nextafter(x, torch.zeros_like(x))], 1)
        q, s = tq.fp8_quantize(x)
        rq, rs = ref_quant_rows(x.double())
        assert torch.equal(s.double(), rs) and _same(q, rq)


def test_zeros_tiny_and_non_finite_blocks(tq):
    import torch
    x = _rng(1)(6, 400).float()
    x[0] = 0
    x[1] = 1e-45
    x[2, 130] = float("nan")
    x[3, 399] = float("-inf")
    x[4, :128] = -0.0
    x[5] = 3.4e38
    q, s = tq.fp8_quantize(x)
    rq, rs = ref_quant_rows(x.double())
    assert (s[:, 0] == 1).all() and (q[0].float() == 0).all()
    assert s[1, 2].isnan() and q[2, 128:256].float().isnan().all() and torch.isfinite(q[2, :128].float()).all()
    assert s[3, 3].isnan() and q[3, 384:].float().isnan().all()
    assert torch.equal(s.nan_to_num().double(), rs.nan_to_num()) and _same(q, rq)


@pytest.mark.parametrize("C", [256, 1000, 100])
def test_gather_padding_and_factors(tq, C):
    import torch
    T, R = 40, 101
    x = _rng(C)(T, C).to(torch.bfloat16)
    rows = torch.randint(0, T, (R,), device="cuda", dtype=torch.int32)
    rows[::7] = -1
    rows[3] = T
    rows[5] = 2 ** 31 - 1
    f = torch.rand(R, device="cuda")
    live = (rows >= 0) & (rows < T)
    q, s = tq.fp8_quantize(x, rows=rows, row_scale=f)
    v = x.float()[rows.clamp(0, T - 1).long()] * f[:, None]     # one fp32 rounding, as the kernel's
    v[~live] = 0
    rq, rs = ref_quant_rows(v.double())
    assert torch.equal(s.double(), rs) and _same(q, rq)


def test_all_padding(tq):
    """Row numbers into an x without rows: zeros, with scales of 1."""
    import torch
    x = torch.empty(0, 384, dtype=torch.bfloat16, device="cuda")
    rows = torch.zeros(11, dtype=torch.int32, device="cuda")
    out = torch.full((11, 384), 3.0, device="cuda").to(torch.float8_e4m3fn)
    q, s = tq.fp8_quantize(x, rows=rows, row_scale=torch.full((11,), float("nan"), device="cuda"), out=out)
    assert (q.float() == 0).all() and (s == 1).all()


def test_rows_strides(tq):
    import torch
    base = _rng(3)(20, 700).to(torch.float16)
    for x in (base[:, 8:8 + 300], base[:, 16:16 + 257]):
        C = x.shape[1]
        big = torch.zeros(20, 331, dtype=torch.float8_e4m3fn, device="cuda")
        sc = torch.full((-(-C // 128), 29), -1.0, device="cuda")
        q, s = tq.fp8_quantize(x, out=big[:, :C], scales=sc[:, :20])
        rq, rs = ref_quant_rows(x.double())
        assert torch.equal(s.double(), rs) and _same(q, rq)
        assert (big[:, C:].float() == 0).all() and (sc[:, 20:] == -1).all()
    with pytest.raises(tq.TileQError):      # a base that is not 16-byte aligned
        tq.fp8_quantize(base[:, 3:])
    with pytest.raises(ValueError):
        tq.fp8_quantize(base, scales=torch.zeros(1, 20, device="cuda").expand(6, 20))


@pytest.mark.parametrize("dtype", ["bfloat16", "float16", "float32"])
@pytest.mark.parametrize("R,C", [(1, 128), (33, 1408), (70, 260), (9, 36)])
def test_swiglu_rows(tq, R, C, dtype):
    """Values in fp32 are within 2^-21 of silu(g) u w: expf 2 units of 2^-23 (halved or less by 1 + e), four more
    roundings of 2^-24.  The result is then off by half an e4m3 step (2^-4 relative, 2^-10 scales at least)."""
    import torch
    r = _rng(R + C)
    x, w = (r(R, 2 * C) * 3).to(getattr(torch, dtype)), torch.rand(R, device="cuda") + 0.1
    q, s = tq.fp8_quantize(x, swiglu=True, row_scale=w)
    g, u = x.double().chunk(2, 1)
    h = g * torch.sigmoid(g) * u * w.double()[:, None]
    sc = s.t().double().repeat_interleave(128, 1)[:, :C]
    eps = 2.0 ** -21
    lim = h.abs() * (2.0 ** -4 * (1 + eps) + eps) + 2.0 ** -10 * sc
    assert ((dequant_rows(q, s) - h).abs() <= lim).all()
    for b in range(s.shape[0]):
        top = h[:, 128 * b:128 * (b + 1)].abs().amax(1)
        lo, hi = block_scale(top * (1 - eps)), block_scale(top * (1 + eps))
        assert ((s[b].double() == lo) | (s[b].double() == hi)).all()


def _check_codes(q, s, h, eps):
    """q and s of values that are h to within eps relative (and 2^-146: subnormal values' few last places): the exact
    code wherever h / scale is further than that from a tie, one of its two neighbours inside; the exact scale wherever
    the block's maximum is further than that from 448 times a power of two.  Returns how many codes had to be exact."""
    import torch
    exact = 0
    for b in range(s.shape[0]):
        at = slice(128 * b, 128 * (b + 1))
        part, sc = h[:, at], s[b].double()
        top = part.abs().amax(1)
        lo, hi = block_scale(top * (1 - eps)), block_scale(top * (1 + eps))
        assert ((sc == lo) | (sc == hi)).all()
        v, off = part / sc[:, None], eps * part.abs() / sc[:, None] + 2.0 ** -146 / sc[:, None]
        below, above = (round_e4m3((v - off).clamp(-448, 448)), round_e4m3((v + off).clamp(-448, 448)))
        got = q[:, at].float().double()
        assert ((got == below) | (got == above)).all()
        exact += int((below == above).sum())
    return exact


# Values in fp32: expf is within 2 units of 2^-23 (CUDA's bound), e in silu = g e / (1 + e) enters with a factor of at
# most 1; 1 + e and g e are rounded (2^-24 each), the quotient is within 2 units, and two more products are rounded
SWIGLU_EPS = 2.0 ** -20      # 6 * 2^-23, rounded up


@pytest.mark.parametrize("gathered", [False, True])
@pytest.mark.parametrize("dtype", ["bfloat16", "float16", "float32"])
def test_swiglu_codes(tq, dtype, gathered):
    """A million values: 2^-12 of error in the arithmetic would change thousands of codes."""
    import torch
    r, T, C = _rng(17), 512, 2048
    x = r(T, 2 * C).to(getattr(torch, dtype)) * 3
    rows = None
    if gathered:
        rows = (torch.rand(T, generator=torch.Generator("cuda").manual_seed(5), device="cuda") * (T + 6) - 3).to(torch.int32)
    w = r(T).abs() + 0.1
    q, s = tq.fp8_quantize(x, rows=rows, swiglu=True, row_scale=w)
    at, live = (torch.arange(T, device="cuda"), None) if rows is None else (rows.clamp(0, T - 1).long(), (rows >= 0) & (rows < T))
    g, u = x[at].double().chunk(2, 1)
    h = g * torch.sigmoid(g) * u * w.double()[:, None]
    if live is not None:
        h[~live] = 0
        assert (s[:, ~live] == 1).all()
    assert _check_codes(q, s, h, SWIGLU_EPS) > 0.999 * h.numel()


@pytest.mark.parametrize("dtype", ["bfloat16", "float16", "float32"])
def test_swiglu_next_to_ties_and_borders(tq, dtype):
    """Row factors that put a value 2^-18 to either side of a tie, or the block's maximum as far from 448 * 2^k: those
    codes and scales are decided, as the arithmetic is within 2^-20."""
    import torch
    r, R, C = _rng(23), 4096, 128
    x = (r(R, 2 * C) * 2).to(getattr(torch, dtype))
    g, u = x.double().chunk(2, 1)
    h = g * torch.sigmoid(g) * u
    top = h.abs().amax(1)
    # the largest value below half of the maximum that is far enough from zero, to be placed on 1.0625 * 2^m
    mid = torch.where(h.abs() < top[:, None] / 2, h.abs(), torch.zeros_like(h)).amax(1)
    assert (mid > top / 64).all()
    side = 1 + torch.sign(r(R)).double() * 2.0 ** -18
    two = torch.exp2((r(R) * 20).round().double())
    for w in (448 * two / top * side, 1.0625 * two / mid * side):
        w = w.float()
        q, s = tq.fp8_quantize(x, swiglu=True, row_scale=w)
        hw = h * w.double()[:, None]
        assert _check_codes(q, s, hw, SWIGLU_EPS) > 0.999 * h.numel()


def test_swiglu_of_tiny_values(tq):
    """Results below the normal range of fp32: nothing is flushed to zero before the block's scale of 2^-126."""
    import torch
    r = _rng(29)
    x = torch.cat([r(64, 256) * 1e-20, r(64, 256) * torch.logspace(-20, -24, 64, device="cuda")[:, None]], 1).float()
    q, s = tq.fp8_quantize(x, swiglu=True)
    g, u = x.double().chunk(2, 1)
    _check_codes(q, s, g * torch.sigmoid(g) * u, SWIGLU_EPS)
    # row k's largest value is some 2.5e-40 * 10^(-k / 16); codes other than zero start at half of 2^-9 * 2^-126, so that
    # the first 22 rows or so have some
    assert (s == 2.0 ** -126).any() and (q.float() != 0).any(1).sum() >= 16


def test_swiglu_far_values(tq):
    """Gates at both ends of the exponential: silu goes to the gate itself and to zero, not to NaN."""
    import torch
    g = torch.tensor([-3e4, -200.0, -90.0, -88.0, 0.0, 88.0, 200.0, 3e4], device="cuda")
    x = torch.cat([g, torch.ones(8, device="cuda")])[None].to(torch.bfloat16)
    q, s = tq.fp8_quantize(x, swiglu=True)
    v = dequant_rows(q, s)[0]
    assert torch.isfinite(v).all() and v[0] == 0 and v[1] == 0 and v[4] == 0
    assert (v[7] - x[0, 7].double()).abs() <= x[0, 7].double() / 16


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("E,O,I", [(1, 128, 128), (3, 200, 500), (2, 16, 4096), (5, 1, 1), (1, 696, 1000)])
def test_weights(tq, E, O, I, dtype):
    import torch
    w = _rng(O)(E, O, I).to(getattr(torch, dtype))
    q, s = tq.fp8_quantize_weights(w)
    rq, rs = ref_quant_weights(w.double())
    assert torch.equal(s.double(), rs) and _same(q, rq)
    q0, s0 = tq.fp8_quantize_weights(w[0])
    assert torch.equal(s0, s[0]) and _same(q0, rq[0])


@pytest.mark.parametrize("dtype", ["bfloat16", "float16", "float32"])
@pytest.mark.parametrize("C", [400, 1024, 2056, 333])
@pytest.mark.parametrize("factor", [False, True])
def test_non_finite_rows_of_every_type(tq, dtype, C, factor):
    """One NaN or infinity anywhere makes its block NaN and leaves the row's others alone: 16-bit rows have a path of
    their own, and a block is the first or the second of a pair."""
    import torch
    dt = getattr(torch, dtype)
    blocks = -(-C // 128)
    x = _rng(C)(6 * blocks, C).to(dt)
    for b in range(blocks):
        for j, v in enumerate((float("nan"), float("inf"), float("-inf"), torch.finfo(dt).max, -torch.finfo(dt).max, 0.0)):
            x[6 * b + j, min(128 * b + 17 * j + 3, C - 1)] = v
    w = torch.full((x.shape[0],), 0.5, device="cuda") if factor else None
    q, s = tq.fp8_quantize(x, row_scale=w)
    rq, rs = ref_quant_rows(x.double() * (0.5 if factor else 1.0))
    assert torch.equal(s.isnan(), rs.isnan()) and torch.equal(s.nan_to_num().double(), rs.nan_to_num())
    for b in range(blocks):
        at = slice(128 * b, 128 * (b + 1))
        bad = s[b].isnan()
        assert int(bad.sum()) == 3
        assert q[bad][:, at].float().isnan().all() and _same(q[~bad][:, at], rq[~bad][:, at])


@pytest.mark.parametrize("dtype", ["float16", "float32"])
@pytest.mark.parametrize("C", [256, 1000, 1027])
def test_factors_of_other_types(tq, C, dtype):
    import torch
    x = _rng(C)(37, C).to(getattr(torch, dtype))
    f = torch.exp(_rng(C + 1)(37))
    q, s = tq.fp8_quantize(x, row_scale=f)
    rq, rs = ref_quant_rows((x.float() * f[:, None]).double())       # one fp32 rounding, as the kernel's
    assert torch.equal(s.double(), rs) and _same(q, rq)


@pytest.mark.parametrize("dtype", ["bfloat16", "float16", "float32"])
@pytest.mark.parametrize("O,I,pad", [(200, 520, 8), (130, 260, 3), (256, 1024, 16), (1, 37, 1)])
def test_weights_strided_and_into_given_arrays(tq, O, I, pad, dtype):
    """Weights inside a larger array, quantised into a larger array, with blocks that are not finite."""
    import torch
    E, dt = 3, getattr(torch, dtype)
    base = _rng(I)(E, O + 2, I + pad).to(dt)
    w = base[:, :O, :I]
    w[1, 0, 0], w[2, O - 1, I - 1] = float("nan"), float("inf")
    big = torch.full((E, O + 1, I + 2 * pad), 3.0, device="cuda").to(torch.float8_e4m3fn)
    sc = torch.full((E + 1, -(-O // 128), -(-I // 128)), -1.0, device="cuda")
    q, s = tq.fp8_quantize_weights(w, out=big[:, :O, :I], scales=sc[:E])
    assert q.data_ptr() == big.data_ptr() and s.data_ptr() == sc.data_ptr()
    rq, rs = ref_quant_weights(torch.where(torch.isfinite(w), w, torch.zeros_like(w)).double())
    bad = torch.zeros_like(s, dtype=torch.bool)
    bad[1, 0, 0] = bad[2, -1, -1] = True
    at = bad.repeat_interleave(128, 1).repeat_interleave(128, 2)[:, :O, :I]
    assert torch.equal(s.isnan(), bad) and torch.equal(q.float().isnan(), at)
    assert torch.equal(s[~bad].double(), rs[~bad]) and torch.equal(q.float().double()[~at], rq[~at])
    assert (big[:, O:].float() == 3).all() and (big[:, :, I:].float() == 3).all() and (sc[E:] == -1).all()


# ------------------------------------------------------------------ products
def _operands(counts, I, O, seed=0, first=0, behind=0):
    """e4m3 operands with scales of any value, not powers of two."""
    import torch
    r = _rng(seed)
    P, E = first + sum(counts) + behind, len(counts)
    I16 = -(-I // 16) * 16
    f8 = torch.float8_e4m3fn
    xq = (r(P, I16) * 60).clamp(-448, 448).to(f8)[:, :I]
    wq = (r(E, O, I16) * 60).clamp(-448, 448).to(f8)[:, :, :I]
    kb = -(-I // 128)
    xs = r(kb, P).exp()
    ws = r(E, -(-O // 128), kb).exp() * 1e-3
    return xq, xs, wq, ws, offsets_of(counts, first, "cuda")


def _check(tq, xq, xs, wq, ws, off, what, **kw):
    y = tq.fp8_gemm(xq, xs, wq, ws, off, **kw)
    assert tq.expert_status() == 0, what
    ref, mag = ref_forward(dequant_rows(xq, xs), dequant_weights(wq, ws), off)
    a, b = int(off[0]), int(off[-1])
    assert_within(y[a:b], ref[a:b], mag[a:b], fp8_terms(xq.shape[1]), what)
    return y


@pytest.mark.parametrize("counts", [FEW, RAGGED, LONG, [1], [1000]], ids=["few", "ragged", "long", "one", "dense"])
@pytest.mark.parametrize("I,O", [(256, 512), (1008, 696), (128, 16), (16, 8), (272, 1032), (2048, 130)])
def test_products(tq, counts, I, O):
    _check(tq, *_operands(counts, I, O), f"{counts} {I} {O}")


@pytest.mark.parametrize("counts,I,O", [([1], 4096, 512), ([7], 2048, 136), ([40], 1104, 264), ([3, 0, 64, 1], 1536, 264),
                                        ([16, 33], 1008, 1000), ([64], 272, 64)])
def test_few_tiles_share_a_reduction(tq, counts, I, O):
    import torch
    ops = _operands(counts, I, O, seed=I)
    y = _check(tq, *ops, f"{counts} {I} {O}")
    assert torch.equal(y, tq.fp8_gemm(*ops))


@pytest.mark.parametrize("out_dtype", ["bfloat16", "float16", "float32"])
def test_product_types_strides_and_other_rows(tq, out_dtype):
    import torch
    dt = getattr(torch, out_dtype)
    counts = [40, 0, 3, 170]
    xq, xs, wq, ws, off = _operands(counts, 200, 52, seed=5, first=6, behind=40)
    xq[:6], xq[-40:] = float("nan"), float("nan")
    xs[:, :6] = float("nan")
    ws = ws * 1e-3                       # results inside fp16's range
    pad = torch.full((xs.shape[0], xs.shape[1] + 5), float("nan"), device="cuda")
    pad[:, 3:-2] = xs
    out = torch.full((xq.shape[0], 67), 9.0, dtype=dt, device="cuda")
    y = _check(tq, xq, pad[:, 3:-2], wq, ws, off, "strides", out=out[:, :52])
    assert (out[:, 52:] == 9).all() and (out[:6] == 9).all() and (out[-40:] == 9).all()
    assert y.dtype == dt


def test_many_tiles_for_every_cta(tq):
    """More tiles than CTAs in the wide kernel; the last column tile has one block of 128, another expert's a part."""
    for O in (1408, 1300):
        _check(tq, *_operands([700, 513, 0, 769, 300, 1025, 257, 640], 656, O, seed=O), f"many tiles {O}")


@pytest.mark.parametrize("counts", [[300], [600, 0, 290], [1024], [128, 140]])
@pytest.mark.parametrize("I,O", [(512, 2048), (640, 1160), (2048, 640)])
def test_shared_tiles_of_a_last_round(tq, counts, I, O):
    """Few wide tiles: two CTAs share each, a part each; the second has nothing to do where d_out ends in the first."""
    _check(tq, *_operands(counts, I, O), "shared")


def test_refusals(tq):
    import torch
    xq, xs, wq, ws, off = _operands([4, 4], 256, 160)
    f = tq.fp8_gemm
    for call in (lambda: f(xq.float(), xs, wq, ws, off), lambda: f(xq, xs.double(), wq, ws, off), lambda: f(xq, xs.t(), wq, ws, off),
                 lambda: f(xq, xs[:1], wq, ws, off), lambda: f(xq, xs[:1].expand(2, 8), wq, ws, off), lambda: f(xq, xs, wq, ws[0], off),
                 lambda: f(xq, xs, wq, ws[:, :1].expand(2, 2, 2), off), lambda: f(xq, xs, wq, ws), lambda: f(xq, xs, wq[0], ws[0], off),
                 lambda: f(xq, xs, wq[:, :, :128], ws[:, :, :1], off), lambda: f(xq, xs, wq, ws, off, out_dtype=torch.float64),
                 lambda: f(xq, xs, wq, ws, off, out=torch.empty(8, 159, dtype=torch.bfloat16, device="cuda"))):
        with pytest.raises(ValueError):
            call()
    x = torch.zeros(8, 257, dtype=torch.bfloat16, device="cuda")
    for call in (lambda: tq.fp8_quantize(x, swiglu=True), lambda: tq.fp8_quantize(x, rows=torch.zeros(4, dtype=torch.int64, device="cuda")),
                 lambda: tq.fp8_quantize(x, row_scale=torch.zeros(7, device="cuda")), lambda: tq.fp8_quantize(x.to(torch.float64)),
                 lambda: tq.fp8_quantize(x, out=torch.zeros(8, 257, device="cuda")), lambda: tq.fp8_quantize_weights(x[None, None]),
                 lambda: tq.fp8_quantize_weights(x, scales=torch.zeros(1, 2, device="cuda"))):
        with pytest.raises(ValueError):
            call()


def test_nan_row_and_nan_weight_block(tq):
    import torch
    xq, xs, wq, ws, off = _operands([20, 300], 384, 300, seed=2)
    xs[1, 7] = float("nan")
    ws[1, 2, 0] = float("inf")
    y = tq.fp8_gemm(xq, xs, wq, ws, off)
    assert y[7].isnan().all() and torch.isfinite(y[[i for i in range(20) if i != 7]]).all()
    assert torch.isfinite(y[20:, :256]).all() and (~torch.isfinite(y[20:, 256:])).all()


@pytest.mark.parametrize("P", [1, 3, 64, 65, 200, 2048])
def test_dense(tq, P):
    xq, xs, wq, ws, off = _operands([P], 640, 392, seed=P)
    import torch
    y = tq.fp8_gemm(xq, xs, wq[0], ws[0])
    assert torch.equal(y, _check(tq, xq, xs, wq, ws, off, "dense"))
    one = _check(tq, xq, xs, wq[:, :1], ws[:, :1], off, "one output")
    assert torch.equal(one, tq.fp8_gemm(xq, xs, wq[0, :1], ws[0, :1]))
    for bad in ((wq[0], ws[0, :, :1]), (wq[0], ws[0].t().contiguous().t()), (wq[0, :0], ws[0, :0]), (wq[0, :, :512], ws[0, :, :4])):
        with pytest.raises(ValueError):
            tq.fp8_gemm(xq, xs, *bad)


def test_no_rows(tq):
    import torch
    xq, xs, wq, ws, off = _operands([0, 0], 128, 64)
    assert tq.fp8_gemm(xq, xs, wq, ws, off).shape == (0, 64)
    q, s = tq.fp8_quantize(torch.zeros(0, 256, dtype=torch.bfloat16, device="cuda"))
    assert q.shape == (0, 256) and s.shape == (2, 0)


def test_same_bits_in_a_graph(tq):
    import torch
    x = _rng(9)(300, 512).to(torch.bfloat16)
    rows = torch.randint(0, 300, (sum(RAGGED),), device="cuda", dtype=torch.int32)
    _, _, wq, ws, off = _operands(RAGGED, 512, 384, seed=4)
    q, s = tq.fp8_quantize(x, rows=rows)
    want = tq.fp8_gemm(q, s, wq, ws, off)
    assert torch.equal(tq.fp8_gemm(q, s, wq, ws, off), want)
    out = torch.zeros_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gq, gs = tq.fp8_quantize(x, rows=rows)
        tq.fp8_gemm(gq, gs, wq, ws, off, out=out)
    for _ in range(3):
        out.zero_()
        graph.replay()
        assert torch.equal(out, want)
    x.copy_(x.roll(1, 0))
    graph.replay()
    q, s = tq.fp8_quantize(x, rows=rows)
    assert torch.equal(out, tq.fp8_gemm(q, s, wq, ws, off))


@pytest.mark.parametrize("out_dtype", ["bfloat16", "float16", "float32"])
@pytest.mark.parametrize("O,pad", [(1290, 1), (1291, 1), (1290, 2), (1304, 8), (1312, 16), (1237, 3)])
def test_wide_tiles_of_every_type_and_stride(tq, O, pad, out_dtype):
    """Experts of many rows, so that the wide tiles are taken: every result type, and rows that allow stores of one, two,
    eight or sixteen values.  What lies around the results, and other experts' NaN, stays where it is."""
    import torch
    dt, I = getattr(torch, out_dtype), 656
    xq, xs, wq, ws, off = _operands(LONG, I, O, seed=O, first=4, behind=5)
    ws = ws * 1e-3                       # results inside fp16's range
    xs[:, :4], xs[:, -5:] = float("nan"), float("nan")
    P = xq.shape[0]
    out = torch.full((P, O + pad), 9.0, dtype=dt, device="cuda")
    y = _check(tq, xq, xs, wq, ws, off, "wide", out=out[:, :O])
    assert y.dtype == dt and (out[:, O:] == 9).all() and (out[:4] == 9).all() and (out[-5:] == 9).all()
