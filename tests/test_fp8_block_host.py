"""Refusals of the FP8 products by blocks and of the norm that need no GPU:
every bad argument is rejected on the host before any HIP call."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

from group_limited_routing_router_amd import moe

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "group_limited_routing_router_amd", "csrc")


@pytest.fixture(scope="module")
def lib():
    return moe.load_library()


def _aligned(offset=0):
    raw = np.zeros(4096, np.uint8)
    return raw, raw.ctypes.data + (-raw.ctypes.data) % 64 + offset


def gemm(**kw):
    d = dict(P=64, S=64, E=4, N=32, K=48, k=1)
    d.update(kw)
    return moe.MoEGemmProblem(*(d[n] for n in ("P", "S", "E", "N", "K", "k")))


def problem(**kw):
    d = dict(T=32, H=256, I=192, E=8, G=4, TG=2, k=2, scale=1.0)
    d.update(kw)
    return moe.MoEProblem(*(d[n] for n in ("T", "H", "I", "E", "G", "TG", "k", "scale")))


BIG = 1 << 40


def gemm_calls(lib, g, p, pairs=None, off=0, dtype=0, accumulate=0, ws=0, n=BIG, **null):
    """The grouped calls with all pointers p, but those named in null."""
    at = lambda name: null.get(name, p)  # noqa: E731
    off, ws = p if off == 0 else off, p if ws == 0 else ws
    return {
        "product": lambda: lib.moe_grouped_gemm_fp8_block(g, at("a"), at("a_scale"), pairs, off, at("w"),
                                                          at("w_scale"), at("out"), dtype, ws, n, None),
        "dgrad": lambda: lib.moe_grouped_gemm_fp8_block_dgrad(g, at("dout"), at("dout_scale"), off, at("w"),
                                                              at("w_scale"), at("da"), dtype, accumulate, ws, n,
                                                              None),
    }


@pytest.mark.parametrize("change,status", [
    (dict(P=-1), 1), (dict(P=1 << 31), 1), (dict(S=-1), 1), (dict(E=0), 1), (dict(k=0), 1), (dict(N=0), 1),
    (dict(N=24), 1), (dict(K=0), 1), (dict(K=24), 1), (dict(E=257), 2), (dict(N=65552), 2), (dict(K=65552), 2),
    (dict(P=1 << 30, S=1 << 30, N=1024, K=1024), 2),
])
def test_gemm_shapes(lib, change, status):
    keep, good = _aligned()
    for name, call in gemm_calls(lib, gemm(**change), good).items():
        assert call() == status, (name, lib.moe_last_error())
        assert lib.moe_last_error()


def test_gemm_pointers(lib):
    keep, good = _aligned()
    keep2, odd = _aligned(8)
    for name, args in (("product", ("a", "a_scale", "w", "w_scale", "out")),
                       ("dgrad", ("dout", "dout_scale", "w", "w_scale", "da"))):
        for arg in args:
            for bad in (None, odd):
                assert gemm_calls(lib, gemm(), good, **{arg: bad})[name]() == 1, (name, arg)
                assert arg.encode() in lib.moe_last_error()
        assert gemm_calls(lib, gemm(), good, off=None)[name]() == 1  # only one expert goes without
        assert gemm_calls(lib, gemm(), good, dtype=7)[name]() == 1
        assert gemm_calls(lib, gemm(P=0, S=0), None)[name]() == 0
    assert gemm_calls(lib, gemm(), good, dtype=1, accumulate=1)["dgrad"]() == 1
    assert gemm_calls(lib, gemm(S=63), good)["product"]() == 1
    assert gemm_calls(lib, gemm(S=0), good, pairs=good)["product"]() == 1
    # a split product needs its workspace
    g = gemm(P=16, S=16, E=1, N=512, K=16384)
    need = moe.moe_gemm_workspace_bytes(g)
    assert need > 0
    for call in gemm_calls(lib, g, good, ws=None).values():
        assert call() == 3
    for call in gemm_calls(lib, g, good, n=need - 1).values():
        assert call() == 3
    for call in gemm_calls(lib, g, good, ws=odd).values():
        assert call() == 3


def test_gathered_codes_past_four_gib(lib):
    keep, good = _aligned()
    S = (0xFFF00000 // 5120) + 1
    assert gemm_calls(lib, gemm(P=64, S=S, K=5120, k=2), good, pairs=good)["product"]() == 2
    assert b"4 GiB" in lib.moe_last_error()
    p = problem(T=S, H=5120)
    ws = moe.moe_fp8_block_workspace_bytes(p)
    assert ws > 0
    assert lib.moe_expert_ffn_fp8_block(p, *[good] * 10, 0, good, ws, None) == 2
    assert lib.moe_forward_fp8_block(p, *[good] * 10, 0, None, None, good, good, ws, None) == 2
    assert lib.moe_expert_gate_up_fp8_block(p, *[good] * 10, None) == 2


def test_quantise(lib):
    keep, good = _aligned()
    keep2, odd = _aligned(4)
    rows = lib.moe_quantize_rows_fp8_block
    for args, status in (((-1, 32), 1), ((1 << 31, 32), 1), ((4, 0), 1), ((4, 24), 1), ((4, 65552), 2)):
        assert rows(*args, good, good, good, None) == status
    assert rows(0, 32, None, None, None, None) == 0
    weights = lib.moe_quantize_weights_fp8_block
    for args, status in (((0, 32, 32), 1), ((257, 32, 32), 2), ((1, 24, 32), 1), ((1, 32, 24), 1), ((1, 65552, 32), 2)):
        assert weights(*args, good, good, good, None) == status
    for i in range(3):
        for bad in (None, odd):
            p = [good] * 3
            p[i] = bad
            assert rows(4, 32, *p, None) == 1 and weights(2, 32, 32, *p, None) == 1
    for C in (-5, 0, 1, 128, 129, 512, 513, 5120, 65536):
        want = 0 if C <= 0 else (-(-C // 128) + 3) // 4 * 4
        assert lib.moe_fp8_block_scales(C) == want


def test_expert_calls(lib):
    keep, good = _aligned()
    keep2, odd = _aligned(8)
    ffn = lambda p, a, dtype=0, ws=good, n=BIG: lib.moe_expert_ffn_fp8_block(p, *a, dtype, ws, n, None)  # noqa: E731
    # x, pairs, offsets, 6 weights, y
    assert ffn(problem(I=100), [good] * 10) == 1 and ffn(problem(H=192), [good] * 10) == 2
    for i in range(10):
        for bad in (None, odd):
            a = [good] * 10
            a[i] = bad
            assert ffn(problem(), a) == 1, i
    assert ffn(problem(), [good] * 10, dtype=3) == 1
    need = moe.moe_fp8_block_workspace_bytes(problem())
    assert ffn(problem(), [good] * 10, ws=None) == 3 and ffn(problem(), [good] * 10, n=need - 1) == 3
    assert ffn(problem(T=0), [None] * 10, ws=None, n=0) == 0
    # x, x_scale, pairs, offsets, 4 weights, h, h_scale
    for i in range(10):
        a = [good] * 10
        a[i] = None
        assert lib.moe_expert_gate_up_fp8_block(problem(), *a, None) == 1, i
    assert lib.moe_expert_gate_up_fp8_block(problem(T=0), *[None] * 10, None) == 0
    # x, pairs, offsets, 6 weights, dy, dx, [dtype], 3 gradients
    back = lambda p, a, b, d0=0, d1=0, acc=0, ws=good, n=BIG: lib.moe_expert_ffn_fp8_block_backward(  # noqa: E731
        p, *a, d0, *b, d1, acc, ws, n, None)
    for i in range(14):
        a = [good] * 14
        a[i] = odd
        assert back(problem(), a[:11], a[11:]) == 1, i
    a, b = [good] * 11, [good] * 3
    assert back(problem(), a, b, d0=2) == 1 and back(problem(), a, b, d1=2) == 1
    assert back(problem(), a, b, d1=1, acc=1) == 1
    assert back(problem(), a, b, n=moe.moe_fp8_block_backward_workspace_bytes(problem()) - 1) == 3
    assert moe.moe_fp8_block_workspace_bytes(problem(G=3)) == 0
    assert moe.moe_fp8_block_backward_workspace_bytes(problem(k=17)) == 0
    # the whole block
    a = [good, good, None] + [good] * 6
    fwd = lambda a, out=good, d=0, y=good, ws=good, n=BIG: lib.moe_forward_fp8_block(  # noqa: E731
        problem(), *a, out, d, None, None, y, ws, n, None)
    for i in (0, 1, 3, 4, 5, 6, 7, 8):
        bad = list(a)
        bad[i] = None
        assert fwd(bad) == 1, i
    assert fwd(a, out=None) == 1 and fwd(a, y=None) == 1 and fwd(a, d=9) == 1 and fwd(a, n=16) == 3


def test_norm(lib):
    keep, good = _aligned()
    keep2, odd = _aligned(8)
    f = ctypes.c_float

    def norm(rows=4, H=64, x=good, xd=0, w=good, b=None, eps=1e-6, out=None, od=0, stats=None):
        return lib.moe_norm(rows, H, x, xd, w, b, f(eps), 0, odd - 8 + 16 if out is None else out, od, stats, None)

    for kw, status in ((dict(rows=-1), 1), (dict(rows=1 << 31), 1), (dict(H=0), 1), (dict(H=12), 1),
                       (dict(H=16392), 2), (dict(x=None), 1), (dict(x=odd), 1), (dict(w=None), 1), (dict(b=odd), 1),
                       (dict(out=odd), 1), (dict(stats=odd), 1), (dict(xd=2), 1), (dict(od=2), 1), (dict(eps=0.0), 1),
                       (dict(eps=float("nan")), 1), (dict(eps=float("inf")), 1), (dict(out=good, od=1), 1)):
        assert norm(**kw) == status, (kw, lib.moe_last_error())
    assert norm(rows=0, x=None, w=None) == 0

    need = moe.moe_norm_workspace_bytes(4, 64)
    assert need == 2 * 64 * 4 and moe.moe_norm_workspace_bytes(4, 12) == 0

    def back(rows=4, H=64, dy=good, dyd=0, x=good, xd=0, w=good, stats=good, dx=good + 16, dxd=0, dw=good, db=None,
             ws=good, n=need):
        return lib.moe_norm_backward(rows, H, dy, dyd, x, xd, w, stats, 0, dx, dxd, dw, db, 0, ws, n, None)

    for kw, status in ((dict(rows=-1), 1), (dict(H=20), 1), (dict(H=16392), 2), (dict(dy=None), 1), (dict(x=odd), 1),
                       (dict(w=None), 1), (dict(stats=None), 1), (dict(dx=odd), 1), (dict(dw=None), 1),
                       (dict(db=odd), 1), (dict(dyd=2), 1), (dict(xd=2), 1), (dict(dxd=2), 1),
                       (dict(dx=good, dxd=1), 1), (dict(ws=None), 3), (dict(ws=odd), 3), (dict(n=need - 1), 3)):
        assert back(**kw) == status, (kw, lib.moe_last_error())


@pytest.mark.parametrize("name", ["moe_fp8.h", "moe_norm.h"])
def test_headers_are_plain_c(tmp_path, name):
    src = tmp_path / "h.c"
    src.write_text(f'#include "{name}"\nint main(void) {{ return 0; }}\n')
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    rocm = os.environ.get("ROCM_PATH", "/opt/rocm")
    subprocess.run(["gcc", "-std=c11", "-Wall", "-Wextra", "-Werror", "-D__HIP_PLATFORM_AMD__", "-fsyntax-only",
                    "-I" + os.path.join(root, "include"), "-I" + os.path.join(rocm, "include"), str(src)], check=True)


def test_scales_on_the_host(tmp_path):
    """csrc/fp8_codes.h compiled for the CPU: for every bf16 magnitude the
    smallest power of two that keeps it within 448."""
    src, so = tmp_path / "s.cpp", tmp_path / "s.so"
    src.write_text('#include "fp8_codes.h"\n'
                   'extern "C" int scale_of(unsigned b) { return moe::fp8_scale_of(b); }\n'
                   'extern "C" unsigned inverse_of(int s) { return moe::fp8_inverse_bits(s); }\n')
    subprocess.run(["g++", "-O2", "-std=c++17", "-Wall", "-Wextra", "-Werror", "-fsanitize=undefined",
                    "-fno-sanitize-recover", "-shared", "-fPIC", "-I", CSRC, "-o", str(so), str(src)], check=True)
    c = ctypes.CDLL(str(so))
    c.inverse_of.restype = ctypes.c_uint
    bits = list(range(0, 0x8000)) + [0x0D7F, 0x0D80, 0x7F7F, 0x7F80, 0x7FC0]
    for b in bits:
        for low in (0, 1, 0xFFFF):
            u = b << 16 | low
            v = float(np.uint32(u).view(np.float32))
            s = c.scale_of(u)
            if not np.isfinite(v) or v < 2.0 ** -100:
                assert s == 127
                continue
            assert v <= 448 * 2.0 ** (s - 127) and v > 448 * 2.0 ** (s - 128), (v, s)
            assert float(np.uint32(c.inverse_of(s)).view(np.float32)) == 2.0 ** (127 - s)
