"""The experts' grouped products on the GPU (forward, both gradients) against their definitions in 64 bits."""
import pytest

from experts_util import assert_within, offsets_of, ref_dw, ref_dx, ref_forward

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


def _make(counts, d_in, d_out, dtype, first=0, behind=0, seed=0):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    off = offsets_of(counts, first, "cuda")
    P, E = first + sum(counts) + behind, len(counts)
    def rnd(*s):
        return torch.randn(*s, generator=g, device="cuda").to(dtype)
    return rnd(P, d_in), rnd(P, d_out), rnd(E, d_out, d_in), off


def _check_all(tq, x, dy, w, off, what):
    y = tq.grouped_gemm(x, w, off)
    dx = tq.grouped_gemm_dx(dy, w, off)
    dw = tq.grouped_gemm_dw(x, dy, off)
    assert tq.expert_status() == 0, what
    a, b = int(off[0]), int(off[-1])
    for name, got, (ref, mag), terms in (("y", y, ref_forward(x, w, off), w.shape[2]),
                                         ("dx", dx, ref_dx(dy, w, off), w.shape[1])):
        assert_within(got[a:b], ref[a:b], mag[a:b], terms, f"{what} {name}")
    ref, mag = ref_dw(x, dy, off)
    assert_within(dw, ref, mag, max(1, int((off[1:] - off[:-1]).max())), f"{what} dw")


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("counts", [FEW, RAGGED, LONG, [1], [1000]], ids=["few", "ragged", "long", "one", "dense"])
@pytest.mark.parametrize("d_in,d_out", [(256, 512), (1000, 696), (64, 16), (8, 8), (264, 1032)])
def test_products(tq, counts, d_in, d_out, dtype):
    import torch
    x, dy, w, off = _make(counts, d_in, d_out, getattr(torch, dtype))
    _check_all(tq, x, dy, w, off, f"{counts} {d_in} {d_out}")


@pytest.mark.parametrize("counts,d_in,d_out", [([1], 4096, 512), ([7], 2048, 136), ([40], 1096, 264), ([3, 0, 64, 1], 1536, 264),
                                               ([16, 33], 712, 1000), ([5], 320, 128), ([64], 136, 64)])
def test_few_tiles_share_a_reduction(tq, counts, d_in, d_out):
    """Calls with so few tiles that CTAs share the sums of one: long reductions, odd parts, some of them empty."""
    import torch
    for dtype in (torch.bfloat16, torch.float16):
        x, dy, w, off = _make(counts, d_in, d_out, dtype, seed=d_in)
        _check_all(tq, x, dy, w, off, f"{counts} {d_in} {d_out}")


@pytest.mark.parametrize("counts", [[4096], [1000, 0, 3, 500], [129, 2000]])
def test_weight_gradient_over_many_rows(tq, counts):
    """dW of small matrices over long sums, which CTAs share."""
    import torch
    x, dy, w, off = _make(counts, 136, 72, torch.bfloat16, seed=11)
    dw = tq.grouped_gemm_dw(x, dy, off)
    ref, mag = ref_dw(x, dy, off)
    assert_within(dw, ref, mag, max(counts), "dw")
    assert torch.equal(dw, tq.grouped_gemm_dw(x, dy, off))


@pytest.mark.parametrize("E", [1, 60, 64, 256])
def test_expert_counts(tq, E):
    import torch
    g = torch.Generator().manual_seed(E)
    counts = torch.randint(0, 40, (E,), generator=g).tolist()
    x, dy, w, off = _make(counts, 136, 200, torch.bfloat16)
    _check_all(tq, x, dy, w, off, f"E={E}")


@pytest.mark.parametrize("counts", [FEW, RAGGED, LONG], ids=["few", "ragged", "long"])
def test_rows_of_no_expert_stay(tq, counts):
    """Rows in front of the first and behind the last expert, NaN in the operands, keep what the output held."""
    import torch
    x, dy, w, off = _make(counts, 192, 320, torch.bfloat16, first=5, behind=70)
    a, b = int(off[0]), int(off[-1])
    for t in (x, dy):
        t[:a] = float("nan")
        t[b:] = float("nan")
    for got in (tq.grouped_gemm(x, w, off, out=torch.full((x.shape[0], 320), 7.0, dtype=x.dtype, device="cuda")),
                tq.grouped_gemm_dx(dy, w, off, out=torch.full((x.shape[0], 192), 7.0, dtype=x.dtype, device="cuda"))):
        assert (got[:a] == 7).all() and (got[b:] == 7).all()
        assert torch.isfinite(got[a:b]).all()
    ref, mag = ref_dw(x, dy, off)
    assert_within(tq.grouped_gemm_dw(x, dy, off), ref, mag, max(counts), "dw")


def test_nan_stays_with_its_expert(tq):
    """A row of NaN and infinities reaches its own row of y and dx and its own expert's dW alone."""
    import torch
    counts = [17, 33, 64, 1, 0, 130, 300]
    x, dy, w, off = _make(counts, 256, 136, torch.bfloat16)
    bad = int(off[2])                      # the row behind expert 1's last one
    x[bad], dy[bad] = float("nan"), float("inf")
    y, dx, dw = tq.grouped_gemm(x, w, off), tq.grouped_gemm_dx(dy, w, off), tq.grouped_gemm_dw(x, dy, off)
    rest = torch.arange(x.shape[0], device="cuda") != bad
    assert y[bad].isnan().all() and torch.isfinite(y[rest]).all()
    assert (~torch.isfinite(dx[bad])).all() and torch.isfinite(dx[rest]).all()
    assert dw[2].isnan().all() and torch.isfinite(dw[[0, 1, 3, 4, 5, 6]]).all()
    assert (dw[4] == 0).all()


@pytest.mark.parametrize("out_dtype", ["bfloat16", "float16", "float32"])
def test_out_types_and_strides(tq, out_dtype):
    """Operands and results inside larger arrays, odd result strides, every result type."""
    import torch
    out_dtype = getattr(torch, out_dtype)
    counts = [40, 0, 3, 170]
    P, E, I, O = sum(counts), 4, 100, 52
    g = torch.Generator(device="cuda").manual_seed(3)
    big = lambda *s: (torch.randn(*s, generator=g, device="cuda") * 0.5).to(torch.bfloat16)  # noqa: E731
    x, dy, w = big(P, 136)[:, 8:8 + I], big(P, 72)[:, 16:16 + O], big(E, 64, 120)[:, 3:3 + O, 8:8 + I]
    off = offsets_of(counts, 0, "cuda")
    y = torch.full((P, 67), 9.0, dtype=out_dtype, device="cuda")[:, :O]
    dx = torch.full((P, 131), 9.0, dtype=out_dtype, device="cuda")[:, :I]
    dw = torch.full((E, O + 3, 113), 9.0, dtype=out_dtype, device="cuda")
    tq.grouped_gemm(x, w, off, out=y)
    tq.grouped_gemm_dx(dy, w, off, out=dx)
    tq.grouped_gemm_dw(x, dy, off, out=dw[:, :O, :I])
    assert_within(y, *ref_forward(x, w, off), I, "y")
    assert_within(dx, *ref_dx(dy, w, off), O, "dx")
    assert_within(dw[:, :O, :I], *ref_dw(x, dy, off), 170, "dw")
    assert (y._base[:, O:] == 9).all() and (dx._base[:, I:] == 9).all()
    assert (dw[:, O:] == 9).all() and (dw[:, :, I:] == 9).all()


def test_widths_without_a_multiple_of_anything(tq):
    import torch
    counts, I, O = [3, 90, 257], 37, 29
    P = sum(counts)
    g = torch.Generator(device="cuda").manual_seed(5)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.float16)  # noqa: E731
    x, dy, w = rnd(P, 40)[:, :I], rnd(P, 32)[:, :O], rnd(3, 29, 40)[:, :, :I]
    _check_all(tq, x, dy, w, offsets_of(counts, 0, "cuda"), "odd widths")
    # one row: its stride is not used, but the rows of w, 37 elements apart, cannot be a tensor map's
    with pytest.raises(tq.TileQError):
        tq.grouped_gemm(rnd(1, I), rnd(1, 2, I), offsets_of([1], 0, "cuda"))


@pytest.mark.parametrize("E", [1, 3])
def test_experts_of_one_output(tq, E):
    """A single row has no row stride that could be unfit."""
    import torch
    x, dy, w, off = _make([5] * E, 40, 1, torch.bfloat16)
    wide = torch.zeros(5 * E, 8, dtype=x.dtype, device="cuda")
    wide[:, :1] = dy
    _check_all(tq, x[:, :37], wide[:, :1], w[:, :, :37], off, "one output")


def test_no_rows(tq):
    import torch
    w = torch.ones(4, 24, 16, dtype=torch.bfloat16, device="cuda")
    x, dy = w.new_empty(0, 16), w.new_empty(0, 24)
    off = offsets_of([0, 0, 0, 0], 0, "cuda")
    assert tq.grouped_gemm(x, w, off).shape == (0, 24) and tq.grouped_gemm_dx(dy, w, off).shape == (0, 16)
    assert (tq.grouped_gemm_dw(x, dy, off) == 0).all()
    # rows, but none of them an expert's
    x, dy = w.new_ones(9, 16), w.new_ones(9, 24)
    out = torch.full((9, 24), 3.0, dtype=w.dtype, device="cuda")
    tq.grouped_gemm(x, w, off, out=out)
    assert (out == 3).all() and (tq.grouped_gemm_dw(x, dy, off) == 0).all()


def test_offsets_out_of_range_are_cut(tq):
    """Bad offsets lead to no access outside the arrays: they are cut to [0, P], a falling one raised."""
    import torch
    x, dy, w, _ = _make([20, 20, 20], 64, 64, torch.bfloat16)
    off = torch.tensor([-5, 20, 10, 4000], dtype=torch.int32, device="cuda")
    cut = torch.tensor([0, 20, 20, 60], dtype=torch.int32, device="cuda")
    assert_within(tq.grouped_gemm(x, w, off), *ref_forward(x, w, cut), 64, "y")
    assert_within(tq.grouped_gemm_dx(dy, w, off), *ref_dx(dy, w, cut), 64, "dx")
    dw = tq.grouped_gemm_dw(x, dy, off)
    assert (dw[1] == 0).all()
    assert_within(dw, *ref_dw(x, dy, cut), 40, "dw")
    assert tq.expert_status() == 0


def test_same_bits_every_time_and_in_a_graph(tq):
    import torch
    x, dy, w, off = _make(RAGGED, 512, 256, torch.bfloat16)
    calls = [lambda **k: tq.grouped_gemm(x, w, off, **k), lambda **k: tq.grouped_gemm_dx(dy, w, off, **k),
             lambda **k: tq.grouped_gemm_dw(x, dy, off, **k)]
    want = [c() for c in calls]
    for c, v in zip(calls, want):
        assert torch.equal(c(), v)
    outs = [torch.zeros_like(v) for v in want]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for c, o in zip(calls, outs):
            c(out=o)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o, v) for o, v in zip(outs, want))
    # another routing of as many rows in the same graph
    other = offsets_of(list(reversed(RAGGED)), 0, "cuda")
    off.copy_(other)
    graph.replay()
    ref, mag = ref_forward(x, w, other)
    assert_within(outs[0], ref, mag, 512, "replayed")
    ref, mag = ref_dw(x, dy, other)
    assert_within(outs[2], ref, mag, max(RAGGED), "replayed dw")


def test_other_streams_at_the_same_time(tq):
    import torch
    a, b = _make(LONG, 256, 384, torch.bfloat16, seed=1), _make(FEW, 384, 256, torch.bfloat16, seed=2)
    want = [tq.grouped_gemm(t[0], t[2], t[3]) for t in (a, b)]
    s = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i, t in enumerate((a, b)):
            got[i].append(tq.grouped_gemm(t[0], t[2], t[3], stream=s[i] if i else s[i].cuda_stream))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want[i]) for i in (0, 1) for o in got[i])


def test_many_tiles_for_every_cta(tq):
    """More tiles than CTAs in the wide kernel, the last of each expert short in both directions."""
    import torch
    x, dy, w, off = _make([700, 513, 0, 769, 300, 1025, 257, 640], 712, 1416, torch.bfloat16, seed=3)
    _check_all(tq, x, dy, w, off, "many tiles")


def test_two_threads_and_two_graphs_at_once(tq):
    import threading

    import torch
    data = [_make(c, 512, 768, torch.bfloat16, seed=i) for i, c in enumerate((LONG, RAGGED))]
    want = [(tq.grouped_gemm(x, w, off), tq.grouped_gemm_dw(x, dy, off)) for x, dy, w, off in data]
    torch.cuda.synchronize()
    got, graphs = [None, None], []
    for x, dy, w, off in data:
        graph, out = torch.cuda.CUDAGraph(), (torch.zeros(x.shape[0], 768, dtype=x.dtype, device="cuda"), torch.zeros_like(w))
        with torch.cuda.graph(graph):
            tq.grouped_gemm(x, w, off, out=out[0])
            tq.grouped_gemm_dw(x, dy, off, out=out[1])
        graphs.append((graph, out))

    def work(i):
        x, dy, w, off = data[i]
        with torch.cuda.stream(torch.cuda.Stream()):
            got[i] = [(tq.grouped_gemm(x, w, off), tq.grouped_gemm_dw(x, dy, off)) for _ in range(30)]
            torch.cuda.current_stream().synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in (0, 1)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for i in (0, 1):
        assert all(torch.equal(a, want[i][0]) and torch.equal(b, want[i][1]) for a, b in got[i])
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(20):
        for (graph, _), s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    for (_, out), v in zip(graphs, want):
        assert torch.equal(out[0], v[0]) and torch.equal(out[1], v[1])


def test_a_first_call_in_a_capture_is_refused(tq, monkeypatch):
    """The device's status word cannot be allocated there; a call before the capture makes it."""
    import torch
    from tiled_rank_b200 import experts
    x, dy, w, off = _make([4, 4], 64, 32, torch.bfloat16)
    with monkeypatch.context() as m:
        m.setattr(experts, "_status_words", {})
        with pytest.raises(RuntimeError, match="outside of the graph"):
            with torch.cuda.graph(torch.cuda.CUDAGraph()):
                tq.grouped_gemm(x, w, off)
    want = tq.grouped_gemm(x, w, off)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = tq.grouped_gemm(x, w, off)
    graph.replay()
    assert torch.equal(y, want)


@pytest.mark.parametrize("counts", [[300], [600, 0, 290], [1024], [128, 140]])
@pytest.mark.parametrize("d_in,d_out", [(512, 2048), (640, 1160), (2048, 640)])
def test_shared_tiles_of_a_last_round(tq, counts, d_in, d_out):
    """Few wide tiles: two pairs share each, an odd number of columns, or none, left for the second."""
    import torch
    x, dy, w, off = _make(counts, d_in, d_out, torch.bfloat16)
    _check_all(tq, x, dy, w, off, "shared")


def test_refusals(tq):
    """What does not fit raises before anything is launched, and the outputs stay as they were."""
    import torch
    x, dy, w, off = _make([4, 4], 64, 32, torch.bfloat16)
    out = torch.full((8, 32), 5.0, dtype=x.dtype, device="cuda")
    f = tq.grouped_gemm
    for call in (lambda: f(x, w, off.long(), out=out), lambda: f(x, w, off[:2], out=out), lambda: f(x, w, off.cpu(), out=out),
                 lambda: f(x, w.half(), off, out=out), lambda: f(x[:, :56], w, off, out=out), lambda: f(x, w[0], off, out=out),
                 lambda: f(x, w.transpose(1, 2), off, out=out), lambda: f(x[:1].expand(8, 64), w, off, out=out),
                 lambda: f(x, w[:1].expand(2, 32, 64), off, out=out), lambda: f(x, w, off, out=out[:7]),
                 lambda: f(x, w, off, out=out.cpu()), lambda: f(x, w, off, out=out, out_dtype=torch.float32),
                 lambda: f(x, w, off, out_dtype=torch.float64), lambda: f(x, w, off, out=out[:1].expand(8, 32)),
                 lambda: f(x.t(), w, off, out=out), lambda: tq.grouped_gemm_dx(x, w, off),
                 lambda: tq.grouped_gemm_dw(x, dy[:7], off), lambda: tq.grouped_gemm_dw(x, dy, off[:1]),
                 lambda: tq.grouped_gemm_dw(x, dy, off, out=torch.empty(2, 64, 32, dtype=x.dtype, device="cuda"))):
        with pytest.raises(ValueError):
            call()
    big = torch.zeros(8, 70, dtype=x.dtype, device="cuda")
    for bad in (big[:, 1:65], big[:, :64]):          # not at 16 bytes; rows 140 bytes apart
        with pytest.raises(tq.TileQError):
            f(bad, w, off, out=out)
    torch.cuda.synchronize()
    assert (out == 5).all()


def test_results_past_2_31_elements(tq):
    """Output offsets that do not fit 32 bits: 70000 x 32768 results, the last rows checked."""
    import torch
    P, I, O = 70000, 64, 32768
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(P, I, generator=g, device="cuda").to(torch.bfloat16)
    w = torch.randn(2, O, I, generator=g, device="cuda").to(torch.bfloat16)
    off = torch.tensor([0, P - 200, P], dtype=torch.int32, device="cuda")
    y = tq.grouped_gemm(x, w, off)
    at = torch.tensor([0, P - 201, P - 200, P - 1], device="cuda")
    e = torch.tensor([0, 0, 1, 1], device="cuda")
    for r, i in zip(at.tolist(), e.tolist()):
        ref, mag = ref_forward(x[r:r + 1], w[i:i + 1], torch.tensor([0, 1]))
        assert_within(y[r:r + 1], ref, mag, I, f"row {r}")


def test_gradients_against_differences(tq):
    """The gradients of sum(y * dy) along random directions against central differences of the forward.

    The forward is bilinear, so a central difference is its derivative but for rounding: with fp32
    results the sum over P * d_out values differs by less than 2^-23 * (d_in + P * d_out) of the
    magnitudes' sum, far under the 1e-3 of the derivative's own scale that is asked for."""
    import torch
    counts, I, O = [30, 0, 100, 270], 64, 48
    x, dy, w, off = _make(counts, I, O, torch.bfloat16, seed=7)
    g = torch.Generator(device="cuda").manual_seed(8)
    # directions and steps that bf16 holds exactly: signs, and operands on a grid of 1/8
    x, w = (x * 8).round().clamp(-16, 16) / 8, (w * 8).round().clamp(-16, 16) / 8
    sign = lambda t: torch.randint(0, 2, t.shape, generator=g, device="cuda").mul_(2).sub_(1).to(t.dtype) / 8  # noqa: E731
    vx, vw = sign(x), sign(w)
    f = lambda a, b: (tq.grouped_gemm(a, b, off, out_dtype=torch.float32).double() * dy.double()).sum()  # noqa: E731
    dx = tq.grouped_gemm_dx(dy, w, off, out_dtype=torch.float32).double()
    dw = tq.grouped_gemm_dw(x, dy, off, out_dtype=torch.float32).double()
    for num, ana, scale in (((f(x + vx, w) - f(x - vx, w)) / 2, (dx * vx.double()).sum(), (dx * vx.double()).norm()),
                            ((f(x, w + vw) - f(x, w - vw)) / 2, (dw * vw.double()).sum(), (dw * vw.double()).norm())):
        assert abs(num - ana) <= 1e-3 * scale, (num, ana, scale)


def test_a_sum_that_takes_longer_than_a_second(tq):
    """One expert of many with 450 million rows: its tile's reduction runs for more than a second, which no bounded wait
    may take for a stop.  Rows of zeros but for three, whose products are small whole numbers."""
    import torch
    P, E, at = 450_000_000, 100, 40
    if torch.cuda.mem_get_info()[0] < 20 << 30:
        pytest.skip("20 GB of device memory")
    x, dy = (torch.zeros(P, 8, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    n = torch.arange(1, 9, device="cuda", dtype=torch.bfloat16)
    for i in (0, P // 2 + 5, P - 1):
        x[i], dy[i] = 1, n
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    off[at + 1:] = P
    dw = tq.grouped_gemm_dw(x, dy, off)
    assert tq.expert_status() == 0
    assert torch.equal(dw[at], (3 * n)[:, None].expand(8, 8))
    assert (dw[:at] == 0).all() and (dw[at + 1:] == 0).all()


def test_results_beside_and_over_operands(tq):
    """Columns of the operands' own rows, the room between them and memory right behind them take a result; a shared
    byte is refused."""
    import torch
    counts, I, O = [40, 0, 3, 170], 64, 48
    x, dy, w, off = _make(counts, I, O, torch.bfloat16, seed=21)
    P, E = sum(counts), len(counts)
    want, wdx, wdw = tq.grouped_gemm(x, w, off), tq.grouped_gemm_dx(dy, w, off), tq.grouped_gemm_dw(x, dy, off)
    both = torch.zeros(P, I + O, dtype=x.dtype, device="cuda")
    both[:, :I] = x
    assert torch.equal(tq.grouped_gemm(both[:, :I], w, off, out=both[:, I:]), want) and torch.equal(both[:, :I], x)
    one = torch.zeros(P * (I + O), dtype=x.dtype, device="cuda")
    a, b = one[:P * I].view(P, I), one[P * I:].view(P, O)
    assert torch.equal(tq.grouped_gemm(a.copy_(x), w, off, out=b), want)
    # a gradient in the columns behind the rows' and behind every matrix of the weights
    rows = torch.zeros(P, O + I, dtype=x.dtype, device="cuda")
    rows[:, :O] = dy
    assert torch.equal(tq.grouped_gemm_dx(rows[:, :O], w, off, out=rows[:, O:]), wdx)
    pair = torch.zeros(E, 2, O, I, dtype=x.dtype, device="cuda")
    pair[:, 0] = w
    assert torch.equal(tq.grouped_gemm(x, pair[:, 0], off), want)
    assert torch.equal(tq.grouped_gemm_dw(x, dy, off, out=pair[:, 1]), wdw) and torch.equal(pair[:, 0], w)
    # results in the gaps of rows of another length
    gaps = torch.zeros(64 * P, dtype=x.dtype, device="cuda")
    xs, ys = gaps.view(P, 64)[:, :16], gaps.view(P // 3, 192)[:, 16:64]
    few = offsets_of([P // 3], 0, "cuda")
    w1 = w[:1, :, :16].contiguous()
    assert torch.equal(tq.grouped_gemm(xs.copy_(x[:, :16])[:P // 3], w1, few, out=ys),
                       tq.grouped_gemm(x[:P // 3, :16].contiguous(), w1, few))
    square = torch.randn(E, I, I, device="cuda").to(x.dtype)
    keep = x.clone()
    for call in (lambda: tq.grouped_gemm(x, square, off, out=x), lambda: tq.grouped_gemm_dx(x, square, off, out=x),
                 lambda: tq.grouped_gemm(both[:, :I], w, off, out=both[:, I - 8:I + O - 8]),
                 lambda: tq.grouped_gemm_dw(x, x[:, :8], off, out=x.view(-1)[:E * 8 * I].view(E, 8, I))):
        with pytest.raises(tq.TileQError):
            call()
    assert torch.equal(x, keep)


@pytest.mark.parametrize("call", ["grouped_gemm", "grouped_gemm_dx", "grouped_gemm_dw", "fp8_quantize",
                                  "fp8_quantize_weights", "fp8_gemm"])
@pytest.mark.parametrize("as_int", [False, True])
def test_operands_dropped_while_another_stream_reads_them(tq, call, as_int):
    """The memory of operands that the caller drops after a call on another stream is not handed out before it has run:
    new tensors of their sizes lie elsewhere, and writing them changes no result."""
    import torch
    counts = [300, 212]
    x, dy, w, off = _make(counts, 512, 1024, torch.bfloat16, seed=31)
    xq, xs = tq.fp8_quantize(x)
    wq, ws = tq.fp8_quantize_weights(w)
    given = {"grouped_gemm": (x, w, off), "grouped_gemm_dx": (dy, w, off), "grouped_gemm_dw": (x, dy, off),
             "fp8_quantize": (x,), "fp8_quantize_weights": (w,), "fp8_gemm": (xq, xs, wq, ws, off)}[call]
    f = getattr(tq, call)
    want = f(*given)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        torch.cuda._sleep(1000)
    f(*given, stream=s)
    # room for all that is made below: asking the driver for memory would wait for the GPU
    room = [torch.empty_like(t) for t in given for _ in range(4)]
    del room
    torch.cuda.synchronize()
    tmp = [t.clone() for t in given]
    at = {t.data_ptr() for t in tmp}
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        torch.cuda._sleep(100_000_000)           # some 50 ms in front of the call
    got = f(*tmp, stream=s.cuda_stream if as_int else s)
    del tmp
    done = s.record_event()
    again = [torch.empty_like(t) for t in given for _ in range(2)]
    assert not done.query()
    assert not at & {t.data_ptr() for t in again}
    for t in again:
        t.view(torch.uint8).fill_(0)
    torch.cuda.synchronize()
    for a, b in zip(got if isinstance(got, tuple) else (got,), want if isinstance(want, tuple) else (want,)):
        assert torch.equal(a.float(), b.float())


def test_autograd_sees_a_given_result_change(tq):
    """A tensor that autograd has saved and a call then writes: its backward pass is refused, not computed from the new
    values.  A call that is refused changes nothing."""
    import torch
    x, dy, w, off = _make([20, 12], 64, 64, torch.bfloat16)
    xq, xs = tq.fp8_quantize(x)
    wq, ws = tq.fp8_quantize_weights(w)
    out = torch.ones(32, 64, device="cuda", dtype=torch.bfloat16)
    given = [out, torch.ones_like(w), torch.ones(1, 32, device="cuda"), torch.ones(2, 1, 1, device="cuda")]
    q, qw = torch.empty_like(xq), torch.empty_like(wq)
    for t, call in ((out, lambda: tq.grouped_gemm(x, w, off, out=out)), (out, lambda: tq.grouped_gemm_dx(dy, w, off, out=out)),
                    (out, lambda: tq.fp8_gemm(xq, xs, wq, ws, off, out=out)),
                    (out, lambda: tq.grouped_gemm(x, w, off, out=out, stream=torch.cuda.Stream())),
                    (given[1], lambda: tq.grouped_gemm_dw(x, dy, off, out=given[1])),
                    (given[2], lambda: tq.fp8_quantize(x, scales=given[2])), (q, lambda: tq.fp8_quantize(x, out=q)),
                    (given[3], lambda: tq.fp8_quantize_weights(w, scales=given[3])),
                    (qw, lambda: tq.fp8_quantize_weights(w[0], out=qw[0]))):
        leaf = torch.ones((), device="cuda", requires_grad=True)
        loss = (leaf * t).sum() if t.dtype != torch.float8_e4m3fn else None
        before = t._version
        call()
        torch.cuda.synchronize()
        assert t._version > before
        if loss is not None:
            with pytest.raises(RuntimeError, match="modified by an inplace operation"):
                loss.backward()
    before = out._version
    with pytest.raises(ValueError):
        tq.grouped_gemm(x, w, off, out=out, out_dtype=torch.float32)
    assert out._version == before
    with torch.inference_mode():                 # no counter to move
        tq.grouped_gemm(x, w, off, out=torch.empty_like(out))


@pytest.mark.parametrize("P", [0, 1, 70, 1500])
def test_one_expert_without_offsets(tq, P):
    import torch
    x, dy, w, off = _make([P], 136, 72, torch.bfloat16, seed=P)
    for f, a, b in ((tq.grouped_gemm, x, w), (tq.grouped_gemm_dx, dy, w), (tq.grouped_gemm_dw, x, dy)):
        want = f(a, b, off)
        assert torch.equal(f(a, b, None), want) and torch.equal(f(a, b, None, stream=torch.cuda.current_stream()), want)
    for f, a in ((tq.grouped_gemm, x), (tq.grouped_gemm_dx, dy)):
        with pytest.raises(ValueError, match="2 experts need expert_offsets"):
            f(a, torch.cat([w, w]), None)


@pytest.mark.parametrize("out_dtype", ["bfloat16", "float16", "float32"])
@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("d_in,d_out,pad", [(1300, 1290, 1), (1300, 1290, 2), (1288, 1304, 8), (1296, 1312, 16), (1111, 1237, 3)])
def test_wide_tiles_of_every_type_and_stride(tq, d_in, d_out, pad, dtype, out_dtype):
    """Experts of many rows, so that the wide tiles are taken, into results inside larger arrays: every result type, and
    rows that allow stores of one, two, eight or sixteen values.  What lies around the results keeps its value."""
    import torch
    dt, out_dt, counts = getattr(torch, dtype), getattr(torch, out_dtype), LONG
    P, E, q = sum(counts) + 9, len(counts), lambda n: -(-n // 8) * 8
    g = torch.Generator(device="cuda").manual_seed(d_in + pad)
    rnd = lambda *s: (torch.randn(*s, generator=g, device="cuda") / 4).to(dt)  # noqa: E731
    x, dy, w = rnd(P, q(d_in))[:, :d_in], rnd(P, q(d_out))[:, :d_out], rnd(E, d_out, q(d_in))[:, :, :d_in]
    off = offsets_of(counts, 4, "cuda")
    a, b = 4, 4 + sum(counts)
    y, dx = (torch.full((P, n + pad), 9.0, dtype=out_dt, device="cuda") for n in (d_out, d_in))
    dw = torch.full((E, d_out + pad, d_in + pad), 9.0, dtype=out_dt, device="cuda")
    tq.grouped_gemm(x, w, off, out=y[:, :d_out])
    tq.grouped_gemm_dx(dy, w, off, out=dx[:, :d_in])
    tq.grouped_gemm_dw(x, dy, off, out=dw[:, :d_out, :d_in])
    for got, (ref, mag), terms, what in ((y[:, :d_out], ref_forward(x, w, off), d_in, "y"),
                                         (dx[:, :d_in], ref_dx(dy, w, off), d_out, "dx")):
        assert_within(got[a:b], ref[a:b], mag[a:b], terms, what)
    assert_within(dw[:, :d_out, :d_in], *ref_dw(x, dy, off), max(counts), "dw")
    for t, n in ((y, d_out), (dx, d_in)):
        assert (t[:, n:] == 9).all() and (t[:a] == 9).all() and (t[b:] == 9).all()
    assert (dw[:, d_out:] == 9).all() and (dw[:, :, d_in:] == 9).all()
    assert tq.expert_status() == 0


def test_a_captured_call_on_a_side_stream(tq):
    """A graph whose calls run on a stream beside the capturing one, with operands that are made and dropped within it."""
    import torch
    x, dy, w, off = _make(LONG, 256, 512, torch.bfloat16, seed=41)
    side, out = torch.cuda.Stream(), torch.empty(x.shape[0], 512, dtype=x.dtype, device="cuda")
    wq, ws = tq.fp8_quantize_weights(w)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        twice = x * 2
        side.wait_stream(torch.cuda.current_stream())
        tq.grouped_gemm(twice, w, off, out=out, stream=side)
        dw = tq.grouped_gemm_dw(twice, dy, off, stream=side)
        q, s = tq.fp8_quantize(twice, stream=side)
        y8 = tq.fp8_gemm(q, s, wq, ws, off, stream=side)
        del twice, q, s
        filler = [torch.zeros_like(x) for _ in range(3)]
        torch.cuda.current_stream().wait_stream(side)
    for _ in range(3):
        for t in (out, dw, y8):
            t.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, tq.grouped_gemm(x * 2, w, off)) and torch.equal(dw, tq.grouped_gemm_dw(x * 2, dy, off))
        assert torch.equal(y8, tq.fp8_gemm(*tq.fp8_quantize(x * 2), wq, ws, off))
        x.copy_(x.roll(1, 0))
    del filler
