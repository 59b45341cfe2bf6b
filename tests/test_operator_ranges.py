"""Sizes next to what 64-bit integers hold, in the host checks of the expert
products and the AdamW step (include/nvfp4.h): refused before any of their
products leaves that range.  CPU only: no pointer is dereferenced, no compute
call is made."""
import ctypes
import os

import pytest

import quantize_precision_gemm_amd as q
from tests.test_operator_checks import ADAMW, FAKE, GROUPED


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(q.lib_path()):
        from quantize_precision_gemm_amd import build as hip_build
        hip_build.build()
    return q.load_library()


MOST = (1 << 31) - 8


@pytest.mark.parametrize("sizes,status", [
    # pass, E, T, N, K: more output tiles than a grid holds
    ((2, 1 << 30, 10, 1 << 25, 1 << 25), -2),  # 2^64 tiles
    ((2, 1 << 29, 10, 1 << 25, 1 << 25), -2),  # 2^63
    ((2, MOST, 10, MOST, MOST), -2), ((0, MOST, MOST, MOST, 64), -2), ((1, MOST, MOST, 64, MOST), -2),
    ((2, 1 << 11, 10, 1 << 8, 1 << 19), -2),   # 2^22, one too many
    ((2, 1 << 11, 10, 1 << 8, (1 << 19) - 256), 0),
    ((0, (1 << 22) - 1, 0, 256, 8), -2), ((0, (1 << 22) - 2, 0, 256, 8), 0),
    ((2, MOST, 10, 0, MOST), 0), ((2, 0, 10, MOST, MOST), 0), ((0, MOST, 10, 0, 8), 0),  # no output
])
def test_grouped_sizes(lib, sizes, status):
    n = ctypes.c_int64(-7)
    assert lib.nvfp4_bf16_grouped_gemm_workspace(*sizes, ctypes.byref(n)) == status
    assert (n.value >= 0) if status == 0 else (n.value == -7)


@pytest.mark.parametrize("n", [(1 << 63) - 1, (1 << 63) - 1024, (1 << 33) + 1, 1 << 62])
def test_adamw_sizes(lib, n):
    t = (q._AdamWTensor * 1)()
    for k in ("p", "g", "m", "v", "m_scale", "v_scale", "copy"):
        setattr(t[0], k, ADAMW[k])
    t[0].n = n
    size = ctypes.c_int64(-7)
    assert lib.nvfp4_adamw_table(t, 1, 1, 1, 8, None, 0, ctypes.byref(size)) == -2 and size.value == -7
    assert lib.nvfp4_adamw(t, 1, 1, 1, 8, 1, 1e-3, 0.9, 0.99, 1e-8, 0.1, FAKE, None, None) == -2
    t[0].n = 1 << 33
    assert lib.nvfp4_adamw_table(t, 1, 1, 1, 8, None, 0, ctypes.byref(size)) == 0 and size.value == 0


@pytest.mark.parametrize("change", [
    {"ldb": 1 << 60, "sb": 0}, {"ldb": (1 << 63) - 8, "sb": (1 << 63) - 8}, {"ldb": 1 << 59, "sb": 0, "N": 16},
    {"pass_": 2, "ldc": 1 << 60, "sc": 0}, {"pass_": 2, "ldc": 1 << 62, "sc": (1 << 63) - 4},
    {"pass_": 2, "ldc": (1 << 63) - 4, "sc": 1 << 62},
    {"pass_": 2, "sc": -(1 << 40)}, {"sb": -(1 << 40)}, {"sb": -64, "N": 0, "lda": 64}, {"pass_": 2, "sc": 60, "N": 8},
])
def test_grouped_strides(lib, change):
    d = dict(GROUPED, **change)
    got = lib.nvfp4_bf16_grouped_gemm(d["pass_"], d["a"], d["lda"], d["b"], d["ldb"], d["sb"], d["ends"], d["E"], d["T"],
                                      d["N"], d["K"], d["c"], d["ldc"], d["sc"], d["dtype"], d["ws"], d["wb"], None)
    assert got == -2
