"""Build libnvfp4.so (HIP, gfx950) in-tree, next to this file.

Flags that matter for results:
  -ffp-contract=off   no fused multiply-add: fp32 scale arithmetic must round
                      after every operation, as the format's definition does;
  packed-fp32-ops off no packed fp32 VALU instructions are generated.
No fast-math: division stays correctly rounded and denormals are kept.
"""
import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libnvfp4.so")
SOURCES = ["api.hip", "quantize.hip", "gemm.hip", "gemm_fp8blk.hip", "gemm_rows.hip", "quantize_i8.hip",
           "adamw.hip", "api_layer.hip", "route.hip", "move_rows.hip", "norm.hip", "linear_backward.hip"]
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
ARCH = "gfx950"

CFLAGS = [
    f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC", "-ffp-contract=off",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall", "-Wno-unused-function",
    "-I", os.path.join(os.path.dirname(HERE), "include"),
]


# Per-source flags.  gemm.hip: the backend's ILP-maximising machine scheduler
# (measured on the NVFP4 GEMM's three 12B-layer passes: +0.7 % fprop, +1.9 %
# dgrad, +2.3 % wgrad, bit-identical outputs).
FILE_FLAGS = {"gemm.hip": ["-mllvm", "--amdgpu-sched-strategy=max-ilp"]}


def _run(cmd, verbose):
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    # the host pass does not know the gfx target feature; that warning is noise
    msg = "\n".join(l for l in (r.stdout + r.stderr).splitlines()
                    if "not a recognized feature for this target" not in l)
    if r.returncode != 0:
        raise RuntimeError(f"build failed: {' '.join(cmd)}\n{msg}")
    if verbose and msg.strip():
        print(msg)


# Host-side AddressSanitizer + UndefinedBehaviorSanitizer build (the C ABI's
# argument validation and dispatch; device code is built as usual, since GPU
# sanitizers are not used here): each -fsanitize= applies to the host pass
# only.  Selected at load time with NVFP4_LIB.
LIB_SAN = os.path.join(HERE, "libnvfp4_san.so")
SAN_FLAGS = ["-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
             "-Xarch_host", "-fno-sanitize-recover=undefined", "-Xarch_host", "-fno-omit-frame-pointer",
             "-Xarch_host", "-g"]


def build(verbose: bool = False, jobs: int = 4, sanitize: bool = False) -> str:
    bdir = BUILD + ("_san" if sanitize else "")
    out = LIB_SAN if sanitize else LIB
    os.makedirs(bdir, exist_ok=True)
    objs = []
    procs = []
    for src in SOURCES:
        obj = os.path.join(bdir, src.replace(".hip", ".o"))
        objs.append(obj)
        cmd = [HIPCC] + CFLAGS + FILE_FLAGS.get(src, []) + (SAN_FLAGS if sanitize else []) + \
            ["-c", os.path.join(CSRC, src), "-o", obj]
        procs.append(cmd)
    # compile in parallel
    from concurrent.futures import ThreadPoolExecutor
    with ThreadPoolExecutor(max_workers=jobs) as ex:
        list(ex.map(lambda c: _run(c, verbose), procs))
    tmp = out + ".tmp"
    link = [HIPCC, f"--offload-arch={ARCH}", "-shared", "-fPIC", "-o", tmp] + objs
    if sanitize:
        link[1:1] = ["-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
                     "-shared-libasan"]
    _run(link, verbose)
    os.replace(tmp, out)
    return out


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv, sanitize="--sanitize" in sys.argv))
