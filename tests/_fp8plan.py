"""The rules of csrc/fp8_plan.h, compiled for the CPU: which tile an FP8 product
runs on, so that a test can say which one it means to reach."""
import ctypes
import functools
import os
import subprocess
import tempfile

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCE = """
#include "fp8_plan.h"
static int pack(const moe::TilePlan& p) { return p.rows | p.nt << 10 | p.splits << 11; }
extern "C" int product(long long P, int E, int N, int K) { return pack(moe::product_plan(P, E, N, K)); }
extern "C" int input_grad(long long P, int E, int N, int K) { return pack(moe::input_grad_plan(P, E, N, K)); }
extern "C" int pair(long long P, int E, int N, int K) { return pack(moe::input_grad_plan(P, E, moe::pair_red(N), K)); }
extern "C" int gated(long long P, int E, int N, int K) { return pack(moe::gated_plan(P, E, N, K)); }
"""


@functools.lru_cache(None)
def _library():
    rocm = os.environ.get("ROCM_PATH", "/opt/rocm")
    with tempfile.TemporaryDirectory() as d:
        src, lib = os.path.join(d, "plan.hip"), os.path.join(d, "plan.so")
        with open(src, "w") as f:
            f.write(SOURCE)
        subprocess.run([os.path.join(rocm, "bin", "hipcc"), "--offload-host-only", "-O1", "-std=c++17", "-shared", "-fPIC",
                        "-I" + os.path.join(ROOT, "group_limited_routing_router_amd", "csrc"),
                        "-I" + os.path.join(ROOT, "include"), src, "-o", lib], check=True)
        return ctypes.CDLL(lib)


def plan(op, P, E, N, K):
    """(rows of the tile, weights past the caches, parts of the reduction) of
    op: product, input_grad, pair (gate's and up's gradients at once) or gated,
    on P positions and weights [E,N,K]."""
    v = getattr(_library(), op)(ctypes.c_longlong(P), E, N, K)
    return v & 1023, bool(v >> 10 & 1), v >> 11
