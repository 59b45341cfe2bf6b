"""Refusals of the expert products, the AdamW step and the int8 linear: the
C ABI's host checks (include/nvfp4.h) reject a bad call before anything is
enqueued, and the binding's checks of tensors raise.  CPU only: no pointer is
dereferenced, no compute call is made."""
import ctypes
import os

import numpy as np
import pytest
import torch

import quantize_precision_gemm_amd as q

FAKE = 0x10000
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(q.lib_path()):
        from quantize_precision_gemm_amd import build as hip_build
        hip_build.build()
    return q.load_library()


GROUPED = dict(pass_=0, a=FAKE, lda=64, b=FAKE, ldb=64, sb=64 * 32, ends=FAKE, E=4, T=10, N=32, K=64, c=FAKE, ldc=64,
               sc=64 * 32, dtype=0, ws=None, wb=0)


@pytest.mark.parametrize("change,status", [
    ({"pass_": 3}, -4), ({"pass_": -1}, -4), ({"dtype": 2}, -4),
    ({"E": -1}, -2), ({"T": -1}, -2), ({"N": 36}, -2), ({"K": 60}, -2), ({"T": 1 << 31}, -2), ({"E": 1 << 31}, -2),
    ({"a": None}, -1), ({"b": None}, -1), ({"c": None}, -1), ({"ends": None}, -1),
    ({"a": FAKE + 2}, -3), ({"b": FAKE + 8}, -3), ({"c": FAKE + 4}, -3), ({"ends": FAKE + 2}, -3),
    ({"c": FAKE + 8, "dtype": 1}, -3),
    ({"lda": 68}, -3), ({"ldb": 76}, -3), ({"ldc": 66}, -3), ({"sb": 64 * 32 + 4}, -3),
    ({"lda": 56}, -2), ({"ldb": 56}, -2), ({"ldc": 28}, -2), ({"sb": 64 * 31}, -2),
    ({"pass_": 1, "lda": 24}, -2), ({"pass_": 1, "ldc": 60}, -2),
    ({"pass_": 2, "sc": 64 * 31}, -2), ({"pass_": 2, "sc": 64 * 32 + 2}, -3),
    ({"T": (1 << 31) - 8, "N": 1 << 20, "ldc": 1 << 20, "sb": 1 << 26}, -2),  # more tiles than a grid holds
    ({"ws": FAKE + 8, "wb": 1 << 20}, -3), ({"ws": FAKE, "wb": -1}, -2),
    ({"lda": 1 << 22}, -2), ({"ldb": 1 << 22, "sb": 1 << 28}, -2),  # rows further apart than 32-bit offsets reach
])
def test_grouped_validation(lib, change, status):
    d = dict(GROUPED, **change)
    got = lib.nvfp4_bf16_grouped_gemm(d["pass_"], d["a"], d["lda"], d["b"], d["ldb"], d["sb"], d["ends"], d["E"], d["T"],
                                      d["N"], d["K"], d["c"], d["ldc"], d["sc"], d["dtype"], d["ws"], d["wb"], None)
    assert got == status


@pytest.mark.parametrize("args,status", [
    ((0, 4, 10, 32, 64), 0), ((3, 4, 10, 32, 64), -4), ((0, -1, 10, 32, 64), -2), ((0, 4, -1, 32, 64), -2),
    ((1, 4, 10, 36, 64), -2), ((2, 4, 10, 32, 60), -2), ((2, 0, 0, 0, 0), 0),
])
def test_grouped_workspace_query(lib, args, status):
    n = ctypes.c_int64(-7)
    assert lib.nvfp4_bf16_grouped_gemm_workspace(*args, ctypes.byref(n)) == status
    assert (n.value >= 0) if status == 0 else (n.value == -7)
    assert lib.nvfp4_bf16_grouped_gemm_workspace(*args, None) == -1


ADAMW = dict(p=FAKE, g=FAKE, m=FAKE, v=FAKE, m_scale=FAKE, v_scale=FAKE, copy=FAKE, n=10, count=1, pd=1, gd=1, bits=8,
             step=1, lr=1e-3, b1=0.9, b2=0.99, eps=1e-8, wd=0.1, gs=FAKE, table=None)


@pytest.mark.parametrize("change,status", [
    ({"pd": 2}, -4), ({"gd": -1}, -4), ({"bits": 16}, -4), ({"count": -1}, -2), ({"step": 0}, -2), ({"n": -1}, -2),
    ({"b1": 1.0}, -4), ({"b1": -0.1}, -4), ({"b2": 1.0}, -4), ({"b2": NAN}, -4), ({"eps": -1e-9}, -4),
    ({"eps": INF}, -4), ({"lr": NAN}, -4), ({"lr": INF}, -4), ({"wd": NAN}, -4),
    ({"p": None}, -1), ({"g": None}, -1), ({"m": None}, -1), ({"v": None}, -1), ({"m_scale": None}, -1),
    ({"v_scale": None}, -1),
    ({"pd": 0}, -4),  # a copy of bf16 parameters
    ({"p": FAKE + 2}, -3), ({"g": FAKE + 2}, -3), ({"copy": FAKE + 1}, -3), ({"m_scale": FAKE + 2}, -3),
    ({"m": FAKE + 2, "bits": 32}, -3), ({"v": FAKE + 1, "bits": 32}, -3), ({"gs": FAKE + 2}, -3),
    ({"table": FAKE + 4}, -3),
    ({"n": 1 << 60}, -2), ({"n": (1 << 33) + 1}, -2),
])
def test_adamw_validation(lib, change, status):
    d = dict(ADAMW, **change)
    t = (q._AdamWTensor * 1)()
    for k in ("p", "g", "m", "v", "m_scale", "v_scale", "copy", "n"):
        setattr(t[0], k, d[k])
    got = lib.nvfp4_adamw(t, d["count"], d["pd"], d["gd"], d["bits"], d["step"], d["lr"], d["b1"], d["b2"], d["eps"],
                          d["wd"], d["gs"], d["table"], None)
    assert got == status


def test_adamw_table(lib):
    """The size, the entries (those with elements) and their first chunks, and its refusals."""
    k = 61
    t = (q._AdamWTensor * k)()
    for i in range(k):
        t[i].n = 0 if i in (0, 7) else 700 * i
        t[i].p = t[i].g = t[i].m = t[i].v = FAKE + 4096 * i
    n = ctypes.c_int64(-7)
    args = (t, k, 1, 1, 32)
    assert lib.nvfp4_adamw_table(*args, None, 0, None) == -1
    assert lib.nvfp4_adamw_table(None, k, 1, 1, 32, None, 0, ctypes.byref(n)) == -1 and n.value == -7
    assert lib.nvfp4_adamw_table(t, k, 1, 1, 16, None, 0, ctypes.byref(n)) == -4 and n.value == -7
    assert lib.nvfp4_adamw_table(t, 48, 1, 1, 32, None, 0, ctypes.byref(n)) == 0 and n.value == 0
    assert lib.nvfp4_adamw_table(*args, None, 0, ctypes.byref(n)) == 0 and n.value == -(-59 * 76 // 8) * 8
    buf = np.full(n.value // 8 + 1, -1, dtype=np.int64)
    assert buf.ctypes.data % 8 == 0
    assert lib.nvfp4_adamw_table(*args, buf.ctypes.data, n.value - 8, ctypes.byref(n)) == -7
    assert lib.nvfp4_adamw_table(*args, buf.ctypes.data + 4, n.value, ctypes.byref(n)) == -3
    assert (buf == -1).all()
    assert lib.nvfp4_adamw_table(*args, buf.ctypes.data, n.value, ctypes.byref(n)) == 0
    entries, first = buf[:59 * 9].reshape(59, 9), buf[59 * 9:].view(np.int32)
    used = [i for i in range(k) if t[i].n]
    chunk = 0
    for row, i in enumerate(used):
        assert entries[row, 0] == t[i].p and entries[row, 7] == t[i].n and first[row] == chunk
        chunk += -(-t[i].n // 1024)
    assert buf[-1] == -1


def test_adamw_null_table_and_empty_calls(lib):
    args = (1, 1, 32, 1, 1e-3, 0.9, 0.99, 1e-8, 0.0, None, None, None)
    assert lib.nvfp4_adamw(None, 1, *args) == -1
    t = (q._AdamWTensor * 3)()  # tensors of no elements need no pointers and launch nothing
    assert lib.nvfp4_adamw(t, 3, *args) in (0, -6)  # (-6: no GPU in this process)


@pytest.mark.parametrize("args,status", [
    # x, rows, cols, ld_x, codes, ld_codes, scales
    ((FAKE, 4, 24, 32, FAKE, 32, FAKE), -2), ((FAKE, -1, 32, 32, FAKE, 32, FAKE), -2),
    ((FAKE, 1 << 31, 32, 32, FAKE, 32, FAKE), -2), ((FAKE, 4, 32, 24, FAKE, 32, FAKE), -2),
    ((FAKE, 4, 32, 32, FAKE, 16, FAKE), -2), ((None, 4, 32, 32, FAKE, 32, FAKE), -1),
    ((FAKE, 4, 32, 32, None, 32, FAKE), -1), ((FAKE, 4, 32, 32, FAKE, 32, None), -1),
    ((FAKE + 8, 4, 32, 32, FAKE, 32, FAKE), -3), ((FAKE, 4, 32, 36, FAKE, 32, FAKE), -3),
    ((FAKE, 4, 32, 32, FAKE + 8, 32, FAKE), -3), ((FAKE, 4, 32, 32, FAKE, 40, FAKE), -3),
    ((FAKE, 4, 32, 32, FAKE, 32, FAKE + 2), -3),
])
def test_i8_quantize_validation(lib, args, status):
    assert lib.nvfp4_i8_quantize(*args, None) == status


I8 = dict(a=FAKE, lda=64, sa=FAKE, b=FAKE, ldb=64, sb=FAKE, M=3, N=5, K=64, c=FAKE, ldc=8, dtype=1)


@pytest.mark.parametrize("change,status", [
    ({"dtype": 3}, -4), ({"M": -1}, -2), ({"N": -1}, -2), ({"K": 40}, -2), ({"K": 1 << 17, "lda": 1 << 17, "ldb": 1 << 17}, -2),
    ({"a": None}, -1), ({"b": None}, -1), ({"c": None}, -1), ({"sa": None}, -1), ({"sb": None}, -1),
    ({"a": FAKE + 8}, -3), ({"b": FAKE + 4}, -3), ({"lda": 72}, -3), ({"ldb": 72}, -3), ({"sa": FAKE + 1}, -3),
    ({"sb": FAKE + 2}, -3), ({"c": FAKE + 8}, -3), ({"c": FAKE + 4, "dtype": 0}, -3), ({"ldc": 6}, -3),
    ({"lda": 48}, -2), ({"ldb": 48}, -2), ({"ldc": 4}, -2), ({"lda": 1 << 23}, -2), ({"ldb": 1 << 23}, -2),
    ({"M": (1 << 31) - 1, "N": (1 << 31) - 4, "ldc": 1 << 31}, -2),
])
def test_i8_gemm_validation(lib, change, status):
    d = dict(I8, **change)
    got = lib.nvfp4_i8_gemm(d["a"], d["lda"], d["sa"], d["b"], d["ldb"], d["sb"], d["M"], d["N"], d["K"], d["c"], d["ldc"],
                            d["dtype"], None)
    assert got == status


def test_binding_refuses_cpu_tensors_and_wrong_types():
    x = torch.zeros(4, 32, dtype=torch.bfloat16)
    ends = torch.tensor([4], dtype=torch.int32)
    with pytest.raises(TypeError):
        q.nvfp4_bf16_grouped_gemm(q.FPROP, x, torch.zeros(1, 8, 32, dtype=torch.bfloat16), ends)
    with pytest.raises(TypeError):
        q.nvfp4_i8_quantize(x)
    i8 = q.I8Tensor(torch.zeros(4, 32, dtype=torch.int8), torch.zeros(4))
    with pytest.raises(TypeError):
        q.nvfp4_i8_gemm(i8, i8)
    with pytest.raises(TypeError):
        q.nvfp4_i8_gemm(x, i8)
    with pytest.raises(TypeError):
        q.nvfp4_adamw([x], 1, 1e-3)
    f = torch.zeros(8)
    with pytest.raises(TypeError):  # not on a GPU
        q.AdamWGroup([f], [f], [f], [f])
    with pytest.raises(ValueError):  # one list too short
        q.AdamWGroup([f], [], [f], [f])
    with pytest.raises(ValueError):  # one of the two lists of scales
        q.AdamWGroup([f], [f], [f], [f], m_scales=[f])
    with pytest.raises(TypeError):
        q.AdamWGroup([f.half()], [f], [f], [f])
    with pytest.raises(ValueError):
        q.AdamWGroup.with_states([f], [f], bits=16)


def test_an_empty_group_does_nothing():
    q.nvfp4_adamw(q.AdamWGroup([], [], [], []), 1, 1e-3)


def test_adamw_table_mirrors_the_header():
    assert ctypes.sizeof(q._AdamWTensor) == 64
    assert q._AdamWTensor.n.offset == 56
