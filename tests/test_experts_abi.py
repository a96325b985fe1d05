"""The experts' products without a GPU: struct layout and every refusal, before anything is launched."""
import ctypes
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CALLS = ("tileq_grouped_gemm", "tileq_grouped_gemm_dx", "tileq_grouped_gemm_dw")
A16, ODD = 0x10000, 0x10008          # addresses the checks look at and nothing reads


@pytest.fixture(scope="module")
def L():
    from tiled_rank_b200 import _lib
    if not os.path.exists(_lib.LIB_PATH):
        from tiled_rank_b200 import build
        build.build()
    return _lib


def test_struct_layout_matches_c(L, tmp_path):
    names = [f[0] for f in L.tileq_grouped._fields_]
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "tileq.h"\nint main(void){printf("%zu", sizeof(tileq_grouped));\n'
                   + "".join(f'printf(" %zu", offsetof(tileq_grouped, {n}));\n' for n in names)
                   + 'printf(" %d %d %d %d %d %d", TILEQ_DT_BF16, TILEQ_DT_F16, TILEQ_DT_F32, TILEQ_DT_E4M3,'
                     ' TILEQ_GROUPED_MAX_E, TILEQ_GROUPED_WS_BYTES);return 0;}\n')
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = [int(v) for v in subprocess.run([str(exe)], capture_output=True, text=True).stdout.split()]
    assert got == [ctypes.sizeof(L.tileq_grouped), *(getattr(L.tileq_grouped, n).offset for n in names),
                   L.TILEQ_DT_BF16, L.TILEQ_DT_F16, L.TILEQ_DT_F32, L.TILEQ_DT_E4M3, L.TILEQ_GROUPED_MAX_E,
                   L.TILEQ_GROUPED_WS_BYTES]


def _call(L, name, ws=A16, ws_bytes=256, a=A16, b=A16, out=A16, **fields):
    g = L.tileq_grouped(0, 0, 4, 32, 64, 128, 0, 0, 0, 0, A16)
    for k, v in fields.items():
        setattr(g, k, v)
    return getattr(L.lib(), name)(ctypes.byref(g), a, b, out, ws, ws_bytes, None)


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("bad", [
    dict(E=0), dict(E=257), dict(P=-1), dict(d_in=0), dict(d_out=0), dict(d_in=-8), dict(dtype=2), dict(dtype=3),
    dict(dtype=-1), dict(out_dtype=3), dict(out_dtype=-1), dict(ld_x=-8), dict(ld_y=-8), dict(ld_w=-8), dict(stride_w=-8),
    dict(ld_x=32), dict(ld_y=64), dict(ld_w=32), dict(stride_w=64), dict(expert_offsets=None), dict(expert_offsets=0x10002),
    dict(a=None), dict(b=None), dict(out=None), dict(ws=None), dict(a=ODD), dict(b=ODD), dict(out=ODD),
])
def test_invalid_arguments(L, name, bad):
    assert _call(L, name, **bad) == L.TILEQ_ERR_INVALID_ARG


@pytest.mark.parametrize("name", CALLS)
def test_null_struct_and_short_workspace(L, name):
    assert getattr(L.lib(), name)(None, A16, A16, A16, A16, 256, None) == L.TILEQ_ERR_INVALID_ARG
    assert _call(L, name, ws_bytes=255) == L.TILEQ_ERR_WORKSPACE


@pytest.mark.parametrize("name,bad", [
    ("tileq_grouped_gemm", dict(ld_x=68)), ("tileq_grouped_gemm", dict(ld_w=68)), ("tileq_grouped_gemm", dict(stride_w=64 * 128 + 4)),
    ("tileq_grouped_gemm", dict(d_in=60)), ("tileq_grouped_gemm_dx", dict(ld_y=132)), ("tileq_grouped_gemm_dx", dict(ld_w=68)),
    ("tileq_grouped_gemm_dw", dict(ld_x=68)), ("tileq_grouped_gemm_dw", dict(ld_y=132)), ("tileq_grouped_gemm_dw", dict(d_out=132)),
    ("tileq_grouped_gemm", dict(ld_x=1 << 40)), ("tileq_grouped_gemm", dict(stride_w=1 << 40)),
])
def test_strides_a_tensor_map_cannot_have(L, name, bad):
    assert _call(L, name, **bad) == L.TILEQ_ERR_UNSUPPORTED


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("field", ["P", "d_in", "d_out"])
def test_sizes_near_the_end_of_the_integers(L, name, field):
    assert _call(L, name, **{field: (1 << 31) - 8}) == L.TILEQ_ERR_UNSUPPORTED


@pytest.mark.parametrize("field", ["d_in", "d_out"])
def test_weights_near_the_end_of_the_integers(L, field):
    g = L.tileq_grouped(0, 0, 4, 0, 64, 128, 0, 0, 0, 0, None)
    setattr(g, field, (1 << 31) - 8)
    assert L.lib().tileq_fp8_quantize_weights(ctypes.byref(g), A16, A16, 0, 0, A16, None) == L.TILEQ_ERR_UNSUPPORTED


@pytest.mark.parametrize("name", CALLS[:2])
def test_no_rows_enqueue_nothing(L, name):
    assert _call(L, name, P=0, a=None, out=None) == L.TILEQ_OK


# ------------------------------------------------------------------ fp8
def test_fp8_rows_layout_matches_c(L, tmp_path):
    names = [f[0] for f in L.tileq_fp8_rows._fields_]
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "tileq.h"\nint main(void){printf("%zu", sizeof(tileq_fp8_rows));\n'
                   + "".join(f'printf(" %zu", offsetof(tileq_fp8_rows, {n}));\n' for n in names) + 'return 0;}\n')
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = [int(v) for v in subprocess.run([str(exe)], capture_output=True, text=True).stdout.split()]
    assert got == [ctypes.sizeof(L.tileq_fp8_rows), *(getattr(L.tileq_fp8_rows, n).offset for n in names)]


def _fp8(L, xq=A16, xs=A16, ld_xs=0, wq=A16, sw=A16, y=A16, ws=A16, ws_bytes=256, **fields):
    g = L.tileq_grouped(L.TILEQ_DT_E4M3, 0, 4, 32, 64, 128, 0, 0, 0, 0, A16)
    for k, v in fields.items():
        setattr(g, k, v)
    return L.lib().tileq_fp8_gemm(ctypes.byref(g), xq, xs, ld_xs, wq, sw, y, ws, ws_bytes, None)


@pytest.mark.parametrize("bad", [
    dict(E=0), dict(E=257), dict(P=-1), dict(d_in=0), dict(d_out=0), dict(dtype=0), dict(dtype=4), dict(out_dtype=3),
    dict(ld_x=-16), dict(ld_x=32), dict(ld_w=32), dict(stride_w=64), dict(expert_offsets=None), dict(xq=None), dict(wq=None),
    dict(y=None), dict(xs=None), dict(sw=None), dict(xs=A16 + 2), dict(sw=A16 + 2), dict(xq=ODD), dict(wq=ODD), dict(y=ODD),
    dict(ld_xs=31), dict(ld_xs=-1), dict(ws=None),
])
def test_fp8_gemm_invalid(L, bad):
    assert _fp8(L, **bad) == L.TILEQ_ERR_INVALID_ARG


def test_fp8_gemm_refusals(L):
    assert _fp8(L, ws_bytes=0) == L.TILEQ_ERR_WORKSPACE
    for bad in (dict(d_in=72), dict(ld_x=72), dict(ld_w=72), dict(stride_w=64 * 128 + 8)):
        assert _fp8(L, **bad) == L.TILEQ_ERR_UNSUPPORTED
    assert _fp8(L, P=0, xq=None, xs=None, y=None) == L.TILEQ_OK


def _quant(L, x=A16, q=A16, s=A16, **fields):
    a = L.tileq_fp8_rows(0, 32, 32, 64, 0, None, None, 0, 0, 0)
    for k, v in fields.items():
        setattr(a, k, v)
    return L.lib().tileq_fp8_quantize(ctypes.byref(a), x, q, s, None)


@pytest.mark.parametrize("bad", [
    dict(dtype=3), dict(dtype=-1), dict(R=-1), dict(T=-1), dict(C=0), dict(swiglu=2), dict(T=31), dict(ld_x=63), dict(ld_x=-1),
    dict(ld_q=63), dict(ld_s=31), dict(swiglu=1, ld_x=127), dict(rows=A16 + 2), dict(row_scale=A16 + 1), dict(x=None),
    dict(q=None), dict(s=None), dict(x=ODD), dict(q=ODD), dict(s=A16 + 2),
])
def test_fp8_quantize_invalid(L, bad):
    assert _quant(L, **bad) == L.TILEQ_ERR_INVALID_ARG


@pytest.mark.parametrize("swiglu", [0, 1])
@pytest.mark.parametrize("C", [65535 * 1024 + 1, (1 << 26) + 8, (1 << 31) - 1])
def test_fp8_quantize_rows_too_wide(L, C, swiglu):
    """A size that the kernel's grid cannot have is unsupported, not invalid."""
    big = dict(x=A16, q=1 << 48, s=1 << 52)
    assert _quant(L, C=C, swiglu=swiglu, **big) == L.TILEQ_ERR_UNSUPPORTED


def test_fp8_quantize_no_rows(L):
    assert _quant(L, R=0, x=None, q=None, s=None) == L.TILEQ_OK
    assert L.lib().tileq_fp8_quantize(None, A16, A16, A16, None) == L.TILEQ_ERR_INVALID_ARG


@pytest.mark.parametrize("bad", [
    dict(dtype=3), dict(E=0), dict(E=257), dict(d_in=0), dict(d_out=0), dict(ld_w=63), dict(stride_w=64 * 127), dict(w=None),
    dict(q=None), dict(s=None), dict(w=ODD), dict(q=ODD), dict(ld_q=63), dict(ld_q=-1), dict(stride_q=64), dict(s=A16 + 2),
])
def test_fp8_quantize_weights_invalid(L, bad):
    g = L.tileq_grouped(0, 0, 4, 0, 64, 128, 0, 0, 0, 0, None)
    a = dict(w=A16, q=A16, ld_q=0, stride_q=0, s=A16)
    for k, v in bad.items():
        if k in a:
            a[k] = v
        else:
            setattr(g, k, v)
    assert L.lib().tileq_fp8_quantize_weights(ctypes.byref(g), a["w"], a["q"], a["ld_q"], a["stride_q"], a["s"],
                                              None) == L.TILEQ_ERR_INVALID_ARG


# ------------------------------------------------------------------ results over operands
@pytest.mark.parametrize("name,over", [(n, over) for n in CALLS for over in (
    dict(out=A16), dict(a=A16 + 32, out=A16), dict(b=A16 + (1 << 20)), dict(expert_offsets=A16 + (4 << 20) + 16),
    dict(ws=A16 + (4 << 20) + 64))])
def test_result_over_an_operand(L, name, over):
    """The result lies over the first operand, its second row, the second operand, the offsets or the status word."""
    apart = dict(a=A16, b=A16 + (1 << 20), out=A16 + (4 << 20), ws=A16 + (8 << 20), expert_offsets=A16 + (9 << 20))
    if over == dict(b=A16 + (1 << 20)):
        over = dict(out=apart["b"])
    assert _call(L, name, **{**apart, **over}) == L.TILEQ_ERR_INVALID_ARG


def test_fp8_results_over_operands(L):
    big = [A16 + (i << 24) for i in range(1, 9)]
    apart = dict(zip(("xq", "xs", "wq", "sw", "y", "ws", "expert_offsets"), big))
    for k in ("xq", "xs", "wq", "sw", "ws", "expert_offsets"):
        assert _fp8(L, **{**apart, "y": apart[k]}) == L.TILEQ_ERR_INVALID_ARG, k
        assert _fp8(L, **{**apart, k: apart["y"] + 16}) == L.TILEQ_ERR_INVALID_ARG, k
    apart = dict(zip(("x", "q", "s", "rows", "row_scale"), big))
    for a, b in (("q", "x"), ("q", "s"), ("q", "rows"), ("q", "row_scale"), ("s", "x"), ("s", "rows"), ("s", "row_scale")):
        assert _quant(L, **{**apart, a: apart[b]}) == L.TILEQ_ERR_INVALID_ARG, (a, b)
        assert _quant(L, **{**apart, b: apart[a] + 16}) == L.TILEQ_ERR_INVALID_ARG, (a, b)
    g = L.tileq_grouped(0, 0, 4, 0, 64, 128, 0, 0, 0, 0, None)
    for w, q, s in ((0, 0, 1), (0, 1, 0), (1, 0, 0)):
        assert L.lib().tileq_fp8_quantize_weights(ctypes.byref(g), big[w], big[q], 0, 0, big[s], None) == L.TILEQ_ERR_INVALID_ARG


def test_shared_memory_against_every_byte(tmp_path):
    """The host's test for a shared byte, over 200000 pairs of small arrays, against their bytes one by one."""
    src = tmp_path / "share.cpp"
    src.write_text(r'''
#include <cstdio>
#include <cstring>
#include <random>
#include "share.cuh"
using namespace tileq;
static char mem[8192];
static void fill(const Memory &m, char *in) {
  for (long long i = 0; i < m.mats; ++i)
    for (long long r = 0; r < m.rows; ++r)
      for (long long c = 0; c < m.width; ++c) in[(const char *)m.base - mem + i * m.stride + r * m.ld + c] = 1;
}
int main() {
  std::mt19937 rng(1);
  auto pick = [&](int lo, int hi) { return lo + (int)(rng() % (unsigned)(hi - lo + 1)); };
  int yes = 0, no = 0;
  for (int n = 0; n < 200000; ++n) {
    Memory m[2];
    const int same = pick(1, 40);
    for (Memory &a : m) {
      a.width = pick(1, 12);
      a.rows = pick(0, 6);
      a.ld = a.width + (pick(0, 2) ? pick(0, 30) : 0);
      if (!pick(0, 1) && same >= a.width) a.ld = same;
      a.mats = pick(0, 2) ? 1 : pick(1, 4);
      a.stride = a.rows ? (a.rows - 1) * a.ld + a.width + pick(0, 60) : 0;
      if (!pick(0, 1) && a.rows) a.stride = a.rows * a.ld;
      a.base = mem + pick(0, 300);
    }
    static char x[8192], y[8192];
    memset(x, 0, sizeof x), memset(y, 0, sizeof y);
    fill(m[0], x), fill(m[1], y);
    bool want = false;
    for (int i = 0; i < 8192; ++i) want |= x[i] && y[i];
    (want ? yes : no)++;
    if (share(m[0], m[1]) != want || share(m[1], m[0]) != want) return std::printf("case %d: %d\n", n, want), 1;
  }
  std::printf("%d %d", yes, no);
}
''')
    exe = tmp_path / "share"
    subprocess.run(["g++", "-std=c++17", "-O1", "-I", os.path.join(ROOT, "tiled_rank_b200", "csrc"), str(src), "-o", str(exe)],
                   check=True)
    run = subprocess.run([str(exe)], capture_output=True, text=True)
    assert run.returncode == 0, run.stdout
    assert min(int(v) for v in run.stdout.split()) > 20000


def test_tensors_that_do_not_fit():
    torch = pytest.importorskip("torch")
    import tiled_rank_b200 as tq
    x, w, off = torch.zeros(8, 64), torch.zeros(2, 16, 64), torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError):
        tq.grouped_gemm(x, w, off)                             # fp32
    with pytest.raises(ValueError):
        tq.grouped_gemm(x.bfloat16(), w.bfloat16(), off)       # not on a GPU
    with pytest.raises(ValueError):
        tq.grouped_gemm_dx(torch.zeros(8, 16).half(), w.half(), off)
    with pytest.raises(ValueError):
        tq.grouped_gemm_dw(x.bfloat16(), torch.zeros(8, 16).bfloat16(), off)
    with pytest.raises(ValueError):
        tq.fp8_quantize(x.bfloat16())
    with pytest.raises(ValueError):
        tq.fp8_quantize_weights(w.bfloat16())
    with pytest.raises(ValueError):
        tq.fp8_gemm(x, x, w, w, off)
    with pytest.raises(AttributeError):
        tq.no_such_product
    assert "grouped_gemm" in dir(tq)


@pytest.mark.parametrize("call", ["grouped_gemm", "grouped_gemm_dx", "grouped_gemm_dw", "fp8_gemm"])
def test_an_operand_that_requires_a_gradient(call):
    """Autograd would lose it without a word: refused while gradients are enabled, before the tensors are looked at."""
    torch = pytest.importorskip("torch")
    import tiled_rank_b200 as tq
    f8, off = torch.float8_e4m3fn, torch.zeros(3, dtype=torch.int32)
    x, dy, w = torch.zeros(8, 64).bfloat16(), torch.zeros(8, 16).bfloat16(), torch.zeros(2, 16, 64).bfloat16()
    xs, ws = torch.zeros(1, 8), torch.zeros(2, 1, 1)
    args = {"grouped_gemm": (x, w, off), "grouped_gemm_dx": (dy, w, off), "grouped_gemm_dw": (x, dy, off),
            "fp8_gemm": (x.to(f8), xs, w.to(f8), ws, off)}[call]
    f = getattr(tq, call)
    wants = [t for t in args if t.dtype in (torch.bfloat16, torch.float32)]
    for t in wants:
        t.requires_grad_()
        with pytest.raises(ValueError, match="requires a gradient"):
            f(*args)
        with torch.no_grad(), pytest.raises(ValueError, match="on the same GPU"):
            f(*args)
        t.requires_grad_(False)
    with pytest.raises(ValueError, match="requires a gradient"):
        f(*args, out=torch.zeros(8, 16, requires_grad=True))


def test_the_package_imports_without_torch():
    """The binding needs torch only when a call is made with tensors."""
    code = ("import sys; sys.modules['torch'] = None; import tiled_rank_b200 as tq; "
            "assert tq.tileq_launch_count() == 0; print('ok')")
    out = subprocess.run([os.sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert out.stdout.strip() == "ok", out.stderr
