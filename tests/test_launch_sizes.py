"""The grids of the layer operators at the ends of what they accept: a launch has
fewer than 2^32 threads, at most 1024 a workgroup, and at most 65536 workgroups in its second dimension.

CPU only.  A child process loads the library behind a few C functions that stand
in for the HIP runtime's launch and device queries and write down each launch, for 256
compute units; no pointer is dereferenced."""
import json
import os
import shutil
import subprocess
import sys

import pytest

import quantize_precision_gemm_amd as q

STAND_IN = r"""
#include <stddef.h>
#include <stdint.h>
typedef struct { uint32_t x, y, z; } dim3_t;
static dim3_t grid_now, block_now;
static size_t shared_now;
static void* stream_now;
uint64_t launches[64][4];
int launch_count;
int __hipPushCallConfiguration(dim3_t g, dim3_t b, size_t shared, void* s)
{ grid_now = g; block_now = b; shared_now = shared; stream_now = s; return 0; }
int __hipPopCallConfiguration(dim3_t* g, dim3_t* b, size_t* shared, void** s)
{ *g = grid_now; *b = block_now; *shared = shared_now; *s = stream_now; return 0; }
int hipLaunchKernel(const void* f, dim3_t g, dim3_t b, void** args, size_t shared, void* s)
{
    (void)f; (void)args; (void)shared; (void)s;
    if (launch_count < 64) {
        launches[launch_count][0] = g.x; launches[launch_count][1] = (uint64_t)g.y * g.z;
        launches[launch_count][2] = (uint64_t)b.x * b.y * b.z; launches[launch_count][3] = (uint64_t)b.y * b.z;
    }
    ++launch_count;
    return 0;
}
int hipGetLastError(void) { return 0; }
int hipGetDevice(int* d) { *d = 0; return 0; }
int hipDeviceGetAttribute(int* v, int what, int d) { (void)what; (void)d; *v = 256; return 0; }
"""

CHILD = r"""
import ctypes, json, sys
stand_in = ctypes.CDLL(sys.argv[1], mode=ctypes.RTLD_GLOBAL)
lib = ctypes.CDLL(sys.argv[2])
count = ctypes.c_int.in_dll(stand_in, "launch_count")
launches = ((ctypes.c_uint64 * 4) * 64).in_dll(stand_in, "launches")
kinds = {"p": ctypes.c_void_p, "i": ctypes.c_int32, "l": ctypes.c_int64, "f": ctypes.c_float, "d": ctypes.c_double}
out = []
for name, types, args in json.load(sys.stdin):
    count.value = 0
    status = getattr(lib, name)(*[kinds[t](a) for t, a in zip(types, args)])
    out.append([status, [list(launches[i]) for i in range(min(count.value, 64))]])
print(json.dumps(out))
"""

P = 1 << 20  # an address that nothing reads
BIG = (1 << 31) - 1


@pytest.fixture(scope="module")
def grids(tmp_path_factory):
    compiler = next((c for c in ("gcc", "cc", "/opt/rocm/llvm/bin/clang") if shutil.which(c)), None)
    if compiler is None:
        pytest.skip("no C compiler")
    if not os.path.exists(q.lib_path()):
        from quantize_precision_gemm_amd import build as hip_build
        hip_build.build()
    at = tmp_path_factory.mktemp("stand_in")
    source, lib = str(at / "stand_in.c"), str(at / "stand_in.so")
    with open(source, "w") as f:
        f.write(STAND_IN)
    subprocess.run([compiler, "-O1", "-shared", "-fPIC", "-o", lib, source], check=True)

    def run(calls):
        r = subprocess.run([sys.executable, "-c", CHILD, lib, q.lib_path()], input=json.dumps(calls), capture_output=True, text=True)
        assert r.returncode == 0, r.stderr
        return json.loads(r.stdout.splitlines()[-1])
    return run


def check(grids, calls, some=True):
    """Every call is taken and launches something (unless not `some`), and every launch fits."""
    for (name, _, args), (status, launches) in zip(calls, grids(calls)):
        assert status == 0, (name, args, status)
        assert launches or not some, (name, args)
        for x, yz, threads, block_yz in launches:
            assert 1 <= threads <= 1024 and block_yz == 1 and 1 <= x and 1 <= yz <= 65536, (name, args, launches)
            assert x * yz * threads < 1 << 32, (name, args, launches)


def linear(T, N, K, E=0, f32=1, ws=0):
    return ["nvfp4_bf16_linear", "pl" "pll" "p" "llll" "pli" "i" "pl" "pl" "pli" "plp",
            [P, max(K, 8), P, max(K, 8), N * max(K, 8), P if E else None, E or 1, T, N, K, P, N, 1, 2, None, 0, None, 0, P, N, f32,
             P if ws else None, ws, None]]


# the largest N that the sizes' check takes for so many dense rows: 2^22 tiles of 256 x 256
def widest(T, E=1):
    return ((1 << 22) - 1) // (T // 256 + E + 1) * 256


@pytest.mark.parametrize("T", [1, 8, 9, 16, 17, 32, 33, 64, 65, 8192])
def test_linear_dense(grids, T):
    widths = [8, 1024, 5120, 1 << 20, 10 ** 8, 178956968, 180 * 10 ** 6, 268435456, widest(T)]
    check(grids, [linear(T, N // 8 * 8, K, f32=f, ws=w) for N in widths if N <= widest(T) for K in (0, 8, 64, 4096) for f in (0, 1)
                  for w in (0, 1 << 30)])


@pytest.mark.parametrize("T,E", [(1, 8), (64, 64), (8192, 8), (16, 100000)])
def test_linear_grouped(grids, T, E):
    check(grids, [linear(T, N // 8 * 8, K, E) for N in (8, 5120, 10 ** 6, widest(T, E)) if N <= widest(T, E) for K in (8, 4096)])


@pytest.mark.parametrize("E,N", [(1, 8), (1, 1 << 24), (8, 5120), (65535, 16320), (65535, 8), (63, 1 << 24)])
def test_linear_backward(grids, E, N):
    check(grids, [["nvfp4_bf16_linear_backward", "pi" "l" "pl" "i" "p" "lll" "pl" "p" "plp",
                   [P, 0, N, P, N, 1, P if E > 1 else None, E, T, N, P, N, dbias, P, 1 << 60, None]]
                  for T in (0, 1, 5, 8192, BIG) for dbias in (P, None) if T or dbias])


@pytest.mark.parametrize("cols", [8, 512, 1 << 14, 1 << 24])
@pytest.mark.parametrize("T,k", [(1, 1), (BIG, 1), (BIG, 64)])
def test_move_rows(grids, T, k, cols):
    check(grids, [
        ["nvfp4_dispatch", "pl" "p" "llll" "pl" "p", [P, cols, P, T, k, cols, BIG, P, cols, None]],
        ["nvfp4_combine", "pil" "l" "pp" "lll" "pl" "pli" "p", [P, 1, cols, BIG, P, P, T, k, cols, P, cols, P, cols, 0, None]],
        ["nvfp4_combine_backward", "pil" "pil" "l" "pp" "lll" "pl" "pp", [P, 0, cols, P, 0, cols, BIG, P, P, T, k, cols, P, cols, P, None]]])


@pytest.mark.parametrize("cols", [16, 256, 512, 1 << 14, 1 << 30])
@pytest.mark.parametrize("rows", [1, 3, BIG])
def test_norm(grids, rows, cols):
    calls = [["nvfp4_rmsnorm", "pil" "pli" "pi" "d" "ll" "pl" "pl" "plp" "p",
              [P, 0, cols, P, cols, 0, P, 1, 1e-6, rows, cols, P, cols, P, cols, codes, cols, scales, None]]
             for codes, scales in ((None, None), (P, P))]
    if cols <= 1 << 14:
        calls += [["nvfp4_rmsnorm_backward", "pil" "pl" "pl" "i" "pi" "d" "ll" "pli" "p" "plp",
                   [P, 0, cols, P, cols, P, cols, 0, P, 1, 1e-6, rows, cols, P, cols, 0, dweight, P, 1 << 60, None]]
                  for dweight in (P, None)]
    check(grids, calls)


@pytest.mark.parametrize("E,groups", [(1, 1), (16, 4), (64, 8), (256, 8), (512, 8), (1024, 64)])
@pytest.mark.parametrize("T", [0, 1, 64, 65, 16385, 1 << 27])
def test_route(grids, T, E, groups):
    k = min(15, E)
    check(grids, [["nvfp4_route", "pil" "lll" "p" "ll" "ii" "f" "pppp" "p" "plp",
                   [P, 1, E, T, E, min(k, E // groups * kept), bias, groups, kept, 1, 1, 1.0, P, P, P, P, P, P, 1 << 60, None]]
                  for bias in (P, None) for kept in {1, groups}] +
                 [["nvfp4_route_backward", "pil" "lll" "pp" "p" "ii" "f" "pli" "p", [P, 1, E, T, E, k, P, P, P, 0, 1, 1.0, P, E, 1, None]]],
          some=T > 0)
