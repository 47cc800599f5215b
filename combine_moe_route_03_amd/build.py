"""Build the gfx950 HIP library libmoe_route.so in-tree with hipcc."""
from __future__ import annotations

import concurrent.futures
import os
import subprocess
import tempfile

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
SRC = os.path.join(PKG, "csrc", "moe_route.hip")
LAYER_SRCS = [os.path.join(PKG, "csrc", name) for name in (
    "moe_balance.hip", "moe_experts.hip", "moe_gate.hip", "moe_matmul.hip", "moe_matmul_grad.hip",
    "moe_combine_grad.hip")]
LIB = os.path.join(PKG, "libmoe_route.so")
BENCH_SRC = os.path.join(PKG, "csrc", "bench_copy.hip")
BENCH_LIB = os.path.join(PKG, "libmoe_bench_copy.so")
INCLUDE = os.path.join(ROOT, "include")

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")

# -packed-fp32-ops: keep the compiler from forming packed fp32 add/mul/fma instructions.
FLAGS = ["--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC", "-Wall",
         "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
         "-I", INCLUDE]


def _run(cmd: list, verbose: bool) -> None:
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.check_call(cmd)


def _compile(src: str, lib: str, verbose: bool, more: tuple = ()) -> str:
    """A library of one source, or of several, which are compiled side by side."""
    tmp = lib + ".tmp"
    if not more:
        _run([HIPCC, *FLAGS, "-shared", src, "-o", tmp], verbose)
    else:
        with tempfile.TemporaryDirectory(prefix="moe_build_") as objects:
            pairs = [(s, os.path.join(objects, os.path.basename(s) + ".o")) for s in (src, *more)]
            with concurrent.futures.ThreadPoolExecutor(min(len(pairs), 8)) as pool:
                list(pool.map(lambda p: _run([HIPCC, *FLAGS, "-c", p[0], "-o", p[1]], verbose), pairs))
            _run([HIPCC, "--offload-arch=gfx950", "-shared", *(o for _, o in pairs), "-o", tmp], verbose)
    os.replace(tmp, lib)
    return lib


def build(verbose: bool = False) -> str:
    """Compile the routing library and the benchmark's copy kernel; returns the library path."""
    _compile(BENCH_SRC, BENCH_LIB, verbose)
    return _compile(SRC, LIB, verbose, tuple(LAYER_SRCS))


if __name__ == "__main__":
    print(build(verbose=True))
