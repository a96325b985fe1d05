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


@pytest.mark.parametrize("name", CALLS[:2])
def test_no_rows_enqueue_nothing(L, name):
    assert _call(L, name, P=0, a=None, out=None) == L.TILEQ_OK


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
    with pytest.raises(AttributeError):
        tq.no_such_product
    assert "grouped_gemm" in dir(tq)


def test_the_package_imports_without_torch():
    """The binding needs torch only when a call is made with tensors."""
    code = ("import sys; sys.modules['torch'] = None; import tiled_rank_b200 as tq; "
            "assert tq.tileq_launch_count() == 0; print('ok')")
    out = subprocess.run([os.sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert out.stdout.strip() == "ok", out.stderr
