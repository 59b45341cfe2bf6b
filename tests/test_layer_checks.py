"""Refusals of routing, dispatch and combine, the norm and the linear layer with
its epilogue: the C ABI's host checks (include/nvfp4.h) reject a bad call before
anything is enqueued, and the binding's checks of tensors raise.  CPU only: no
pointer is dereferenced, no compute call is made."""
import ctypes
import os

import pytest
import torch

import quantize_precision_gemm_amd as q

FAKE = 0x10000
NAN, INF = float("nan"), float("inf")
BIG = 1 << 31


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(q.lib_path()):
        from quantize_precision_gemm_amd import build as hip_build
        hip_build.build()
    return q.load_library()


ROUTE = dict(logits=FAKE, ldt=1, ld=64, T=100, E=64, k=4, bias=FAKE, groups=8, kept=2, score=0, renorm=1, scale=1.0,
             experts=FAKE, weights=FAKE, rows=FAKE, ends=FAKE, scores=FAKE, ws=FAKE, wb=1 << 20)


@pytest.mark.parametrize("change,status", [
    ({"ldt": 2}, -4), ({"score": 2}, -4), ({"score": -1}, -4), ({"renorm": 2}, -4), ({"scale": NAN}, -4), ({"scale": INF}, -4),
    ({"T": -1}, -2), ({"T": (1 << 27) + 1}, -2), ({"E": 0}, -2), ({"E": 1025, "ld": 2048}, -2), ({"k": 0}, -2), ({"k": 17}, -2),
    ({"E": 8, "k": 9, "groups": 1, "kept": 1}, -2), ({"ld": 60}, -2), ({"T": 1 << 27, "k": 16}, -2),
    ({"groups": 0}, -2), ({"groups": 7}, -2), ({"groups": 128, "E": 128, "ld": 128}, -2), ({"kept": 0}, -2), ({"kept": 9}, -2),
    ({"kept": 1, "k": 9}, -2), ({"wb": -1}, -2),
    ({"logits": None}, -1), ({"experts": None}, -1), ({"weights": None}, -1), ({"rows": None}, -1), ({"ends": None}, -1),
    ({"logits": FAKE + 2}, -3), ({"logits": FAKE + 1, "ldt": 0}, -3), ({"bias": FAKE + 2}, -3), ({"experts": FAKE + 1}, -3),
    ({"weights": FAKE + 2}, -3), ({"rows": FAKE + 2}, -3), ({"ends": FAKE + 3}, -3), ({"scores": FAKE + 2}, -3), ({"ws": FAKE + 8}, -3),
    ({"ws": None}, -7), ({"wb": 127}, -7), ({"T": 20000, "wb": 313 * 64 + 314 * 64 * 4 - 1}, -7),
])
def test_route_validation(lib, change, status):
    d = dict(ROUTE, **change)
    assert lib.nvfp4_route(d["logits"], d["ldt"], d["ld"], d["T"], d["E"], d["k"], d["bias"], d["groups"], d["kept"], d["score"],
                           d["renorm"], d["scale"], d["experts"], d["weights"], d["rows"], d["ends"], d["scores"], d["ws"],
                           d["wb"], None) == status


@pytest.mark.parametrize("T,E,want", [(0, 64, 0), (64, 64, 0), (65, 64, 2 * 64), (16384, 200, 256 * 256),
                                      (16385, 256, 257 * 256 + 258 * 256 * 4)])
def test_route_workspace(T, E, want):
    assert q.nvfp4_route_workspace(T, E) == want


@pytest.mark.parametrize("T,E", [(-1, 8), ((1 << 27) + 1, 8), (8, 0), (8, 1025)])
def test_route_workspace_refusals(lib, T, E):
    n = ctypes.c_int64(-7)
    assert lib.nvfp4_route_workspace(T, E, ctypes.byref(n)) == -2 and n.value == -7
    assert lib.nvfp4_route_workspace(8, 8, None) == -1


BACK = dict(logits=FAKE, ldt=1, ld=64, T=100, E=64, k=4, experts=FAKE, dw=FAKE, ds=FAKE, score=0, renorm=1, scale=1.0, out=FAKE,
            ldo=64, odt=1)


@pytest.mark.parametrize("change,status", [
    ({"ldt": 3}, -4), ({"odt": 2}, -4), ({"score": 5}, -4), ({"scale": NAN}, -4), ({"k": 17}, -2), ({"ldo": 63}, -2), ({"E": 0}, -2),
    ({"logits": None}, -1), ({"experts": None}, -1), ({"dw": None}, -1), ({"out": None}, -1),
    ({"experts": FAKE + 2}, -3), ({"dw": FAKE + 1}, -3), ({"ds": FAKE + 2}, -3), ({"out": FAKE + 2}, -3), ({"out": FAKE + 1, "odt": 0}, -3),
])
def test_route_backward_validation(lib, change, status):
    d = dict(BACK, **change)
    assert lib.nvfp4_route_backward(d["logits"], d["ldt"], d["ld"], d["T"], d["E"], d["k"], d["experts"], d["dw"], d["ds"], d["score"],
                                    d["renorm"], d["scale"], d["out"], d["ldo"], d["odt"], None) == status


MOVE = dict(x=FAKE, xd=0, ldx=64, o=FAKE, od=0, ldo=64, R=40, rows=FAKE, w=FAKE, T=10, k=4, cols=64, r=FAKE, ldr=64, y=FAKE, ldy=64,
            yd=0, dw=FAKE)
SIZES = [({"T": -1}, -2), ({"T": BIG}, -2), ({"k": 0}, -2), ({"k": 65}, -2), ({"cols": 60}, -2), ({"cols": -8}, -2), ({"R": -1}, -2),
         ({"R": BIG}, -2), ({"cols": (1 << 24) + 8, "ldx": 1 << 26, "ldo": 1 << 26, "ldy": 1 << 26, "ldr": 1 << 26}, -2),
         ({"rows": None}, -1), ({"rows": FAKE + 2}, -3), ({"y": FAKE + 8}, -3), ({"ldy": 56}, -2), ({"ldy": 68}, -3), ({"y": None}, -1)]


@pytest.mark.parametrize("change,status", SIZES + [({"x": None}, -1), ({"x": FAKE + 2}, -3), ({"ldx": 56}, -2), ({"ldx": 68}, -3)])
def test_dispatch_validation(lib, change, status):
    d = dict(MOVE, **change)
    assert lib.nvfp4_dispatch(d["x"], d["ldx"], d["rows"], d["T"], d["k"], d["cols"], d["R"], d["y"], d["ldy"], None) == status


@pytest.mark.parametrize("change,status", SIZES + [
    ({"od": 2}, -4), ({"yd": 2}, -4), ({"o": None}, -1), ({"o": FAKE + 4}, -3), ({"ldo": 56}, -2), ({"ldo": 68}, -3), ({"w": FAKE + 2}, -3),
    ({"r": FAKE + 4}, -3), ({"ldr": 56}, -2), ({"ldr": 66}, -3), ({"ldr": 66, "yd": 1}, -3)])
def test_combine_validation(lib, change, status):
    d = dict(MOVE, **change)
    assert lib.nvfp4_combine(d["o"], d["od"], d["ldo"], d["R"], d["rows"], d["w"], d["T"], d["k"], d["cols"], d["r"], d["ldr"], d["y"],
                             d["ldy"], d["yd"], None) == status


@pytest.mark.parametrize("change,status", SIZES + [
    ({"xd": 2}, -4), ({"od": 7}, -4), ({"x": None}, -1), ({"o": None}, -1), ({"w": None}, -1), ({"dw": None}, -1), ({"dw": FAKE + 2}, -3),
    ({"w": FAKE + 1}, -3), ({"o": FAKE + 4}, -3), ({"ldo": 56}, -2), ({"ldx": 56}, -2)])
def test_combine_backward_validation(lib, change, status):
    d = dict(MOVE, **change)
    assert lib.nvfp4_combine_backward(d["x"], d["xd"], d["ldx"], d["o"], d["od"], d["ldo"], d["R"], d["rows"], d["w"], d["T"], d["k"],
                                      d["cols"], d["y"], d["ldy"], d["dw"], None) == status


NORM = dict(x=FAKE, xd=0, ldx=64, r=FAKE, ldr=64, sd=0, w=FAKE, wd=1, eps=1e-6, rows=5, cols=64, h=FAKE, ldh=64, y=FAKE, ldy=64,
            codes=FAKE, ldc=64, scales=FAKE)


@pytest.mark.parametrize("change,status", [
    ({"xd": 2}, -4), ({"sd": -1}, -4), ({"wd": 3}, -4), ({"eps": -1e-9}, -4), ({"eps": NAN}, -4), ({"eps": INF}, -4),
    ({"rows": -1}, -2), ({"rows": BIG}, -2), ({"cols": 60}, -2), ({"cols": 56}, -2), ({"cols": -16}, -2),
    ({"x": None}, -1), ({"y": None, "codes": None, "scales": None}, -1), ({"codes": None}, -1), ({"scales": None}, -1),
    ({"x": FAKE + 8}, -3), ({"r": FAKE + 8}, -3), ({"h": FAKE + 8}, -3), ({"y": FAKE + 8}, -3), ({"codes": FAKE + 8}, -3),
    ({"scales": FAKE + 2}, -3), ({"w": FAKE + 4}, -3), ({"ldx": 68}, -3), ({"ldr": 68}, -3), ({"ldh": 68}, -3), ({"ldy": 68}, -3),
    ({"ldc": 72}, -3), ({"ldx": 56}, -2), ({"ldr": 56}, -2), ({"ldh": 56}, -2), ({"ldy": 56}, -2), ({"ldc": 48}, -2),
])
def test_rmsnorm_validation(lib, change, status):
    d = dict(NORM, **change)
    assert lib.nvfp4_rmsnorm(d["x"], d["xd"], d["ldx"], d["r"], d["ldr"], d["sd"], d["w"], d["wd"], d["eps"], d["rows"], d["cols"],
                             d["h"], d["ldh"], d["y"], d["ldy"], d["codes"], d["ldc"], d["scales"], None) == status


NORMB = dict(dy=FAKE, dd=0, ldd=64, h=FAKE, ldh=64, dh=FAKE, ldg=64, sd=0, w=FAKE, wd=1, eps=1e-6, rows=5, cols=64, dx=FAKE, ldx=64,
             xd=0, dw=FAKE, ws=FAKE, wb=1 << 30)


@pytest.mark.parametrize("change,status", [
    ({"dd": 2}, -4), ({"sd": 2}, -4), ({"wd": 2}, -4), ({"xd": 2}, -4), ({"eps": NAN}, -4), ({"rows": -1}, -2), ({"cols": 60}, -2),
    ({"cols": 16392, "ldd": 1 << 15, "ldh": 1 << 15, "ldg": 1 << 15, "ldx": 1 << 15}, -2), ({"wb": -1}, -2),
    ({"dy": None}, -1), ({"h": None}, -1), ({"dx": None}, -1), ({"dy": FAKE + 8}, -3), ({"h": FAKE + 8}, -3), ({"dh": FAKE + 8}, -3),
    ({"dx": FAKE + 8}, -3), ({"dw": FAKE + 4}, -3), ({"ws": FAKE + 8}, -3), ({"ldd": 56}, -2), ({"ldh": 56}, -2), ({"ldg": 56}, -2),
    ({"ldx": 56}, -2), ({"ldx": 60, "cols": 56}, -3), ({"rows": 1000, "ws": None}, -7), ({"rows": 1000, "wb": 64}, -7),
])
def test_rmsnorm_backward_validation(lib, change, status):
    d = dict(NORMB, **change)
    assert lib.nvfp4_rmsnorm_backward(d["dy"], d["dd"], d["ldd"], d["h"], d["ldh"], d["dh"], d["ldg"], d["sd"], d["w"], d["wd"],
                                      d["eps"], d["rows"], d["cols"], d["dx"], d["ldx"], d["xd"], d["dw"], d["ws"], d["wb"],
                                      None) == status


LINEAR = dict(x=FAKE, ldx=64, w=FAKE, ldw=64, sw=64 * 32, ends=FAKE, E=4, T=10, N=32, K=64, bias=FAKE, sb=32, bd=1, act=1, r=FAKE,
              ldr=32, pre=FAKE, ldp=32, c=FAKE, ldc=32, cd=0, ws=None, wb=0)


@pytest.mark.parametrize("change,status", [
    ({"cd": 2}, -4), ({"bd": 2}, -4), ({"act": 4}, -4), ({"act": -1}, -4), ({"E": -1}, -2), ({"T": -1}, -2), ({"N": 36}, -2),
    ({"K": 60}, -2), ({"T": BIG}, -2), ({"ends": None}, -2), ({"wb": -1}, -2),
    ({"x": None}, -1), ({"w": None}, -1), ({"c": None}, -1),
    ({"x": FAKE + 8}, -3), ({"w": FAKE + 8}, -3), ({"c": FAKE + 4}, -3), ({"c": FAKE + 8, "cd": 1}, -3), ({"ends": FAKE + 2}, -3),
    ({"bias": FAKE + 8}, -3), ({"bias": FAKE + 4, "bd": 0}, -3), ({"sb": 34}, -3), ({"r": FAKE + 4}, -3), ({"r": FAKE + 8, "cd": 1}, -3),
    ({"ldr": 34}, -3), ({"pre": FAKE + 4}, -3), ({"ldp": 34}, -3), ({"ldx": 68}, -3), ({"ldw": 68}, -3), ({"ldc": 34}, -3),
    ({"sw": 64 * 32 + 4}, -3), ({"ws": FAKE + 8}, -3), ({"ldx": 56}, -2), ({"ldw": 56}, -2), ({"ldc": 28}, -2), ({"ldr": 28}, -2),
    ({"ldp": 28}, -2), ({"sw": 64 * 31}, -2), ({"sb": 28}, -2), ({"ldx": 1 << 22}, -2), ({"ldw": 1 << 22, "sw": 1 << 28}, -2),
    ({"T": BIG - 8, "N": 1 << 20, "ldc": 1 << 20, "ldr": 1 << 20, "ldp": 1 << 20, "sw": 1 << 26, "sb": 1 << 20}, -2),
])
def test_linear_validation(lib, change, status):
    d = dict(LINEAR, **change)
    assert lib.nvfp4_bf16_linear(d["x"], d["ldx"], d["w"], d["ldw"], d["sw"], d["ends"], d["E"], d["T"], d["N"], d["K"], d["bias"],
                                 d["sb"], d["bd"], d["act"], d["r"], d["ldr"], d["pre"], d["ldp"], d["c"], d["ldc"], d["cd"], d["ws"],
                                 d["wb"], None) == status


LINB = dict(dy=FAKE, dd=0, ldd=32, pre=FAKE, ldp=32, act=1, ends=FAKE, E=4, T=10, N=32, out=FAKE, ldo=32, db=FAKE, ws=FAKE, wb=1 << 20)


@pytest.mark.parametrize("change,status", [
    ({"dd": 2}, -4), ({"act": 4}, -4), ({"E": -1}, -2), ({"E": 65536}, -2), ({"T": -1}, -2), ({"T": BIG}, -2), ({"N": 36}, -2),
    ({"N": (1 << 24) + 8, "ldd": 1 << 25, "ldp": 1 << 25, "ldo": 1 << 25}, -2), ({"E": 65535, "N": 16392, "ldd": 16392, "ldp": 16392, "ldo": 16392}, -2),
    ({"wb": -1}, -2), ({"pre": None}, -1), ({"ends": None}, -1), ({"dy": None}, -1), ({"out": None}, -1),
    ({"pre": None, "act": 0, "db": None}, -1), ({"dy": FAKE + 8}, -3), ({"pre": FAKE + 8}, -3), ({"out": FAKE + 8}, -3),
    ({"db": FAKE + 4}, -3), ({"ws": FAKE + 4}, -3), ({"ends": FAKE + 1}, -3), ({"ldd": 24}, -2), ({"ldp": 24}, -2), ({"ldo": 24}, -2),
    ({"ldd": 36}, -3), ({"ldp": 36}, -3), ({"ldo": 36}, -3), ({"ws": None}, -7), ({"wb": 100}, -7),
])
def test_linear_backward_validation(lib, change, status):
    d = dict(LINB, **change)
    assert lib.nvfp4_bf16_linear_backward(d["dy"], d["dd"], d["ldd"], d["pre"], d["ldp"], d["act"], d["ends"], d["E"], d["T"], d["N"],
                                          d["out"], d["ldo"], d["db"], d["ws"], d["wb"], None) == status


@pytest.mark.parametrize("query,good,bad", [
    ("nvfp4_rmsnorm_backward_workspace", (1000, 64), [(-1, 64), (5, 60), (5, 16392), (BIG, 64)]),
    ("nvfp4_bf16_linear_backward_workspace", (4, 10, 32), [(-1, 10, 32), (65536, 10, 32), (4, -1, 32), (4, 10, 36)]),
])
def test_workspace_queries(lib, query, good, bad):
    n = ctypes.c_int64(-7)
    f = getattr(lib, query)
    assert f(*good, None) == -1
    for args in bad:
        assert f(*args, ctypes.byref(n)) == -2 and n.value == -7
    assert f(*good, ctypes.byref(n)) == 0 and n.value > 0 and n.value % 16 == 0


def test_binding_refuses_cpu_tensors_and_wrong_types():
    x, f = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(4, 64)
    places = torch.zeros(4, 2, dtype=torch.int32)
    for call in (lambda: q.nvfp4_route(f, 2), lambda: q.nvfp4_route_backward(f, places, torch.zeros(4, 2)),
                 lambda: q.nvfp4_dispatch(x, places), lambda: q.nvfp4_combine(x, places),
                 lambda: q.nvfp4_combine_backward(x, x, places, torch.zeros(4, 2)), lambda: q.nvfp4_rmsnorm(x),
                 lambda: q.nvfp4_rmsnorm(None), lambda: q.nvfp4_rmsnorm_i8(x), lambda: q.nvfp4_rmsnorm_i8(x, out=x),
                 lambda: q.nvfp4_rmsnorm_backward(x, x), lambda: q.nvfp4_bf16_linear(x, x),
                 lambda: q.nvfp4_bf16_linear_backward(x, x, q.ACT_SILU)):
        with pytest.raises(TypeError):
            call()
