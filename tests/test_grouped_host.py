"""Refusals of the grouped products that need no GPU: every bad argument is
rejected on the host before any HIP call, and the binding's own checks."""
import ctypes

import numpy as np
import pytest
import torch

from group_limited_routing_router_amd import moe


@pytest.fixture(scope="module")
def lib():
    return moe.load_library()


def gemm(**kw):
    d = dict(P=64, S=64, E=4, N=32, K=48, k=1)
    d.update(kw)
    return moe.MoEGemmProblem(*(d[n] for n in ("P", "S", "E", "N", "K", "k")))


def _aligned(offset=0):
    raw = np.zeros(4096, np.uint8)
    return raw, raw.ctypes.data + (-raw.ctypes.data) % 64 + offset


def calls(lib, g, ptr, pairs=None, dtype=0, accumulate=0, off=None, ws=None):
    """Every grouped call on g with all pointers ptr."""
    off = ptr if off is None else off
    n = 1 << 40 if ws else 0
    return {
        "gemm": lambda: lib.moe_grouped_gemm(g, ptr, pairs, off, ptr, ptr, dtype, ws, n, None),
        "dgrad": lambda: lib.moe_grouped_gemm_dgrad(g, ptr, off, ptr, ptr, dtype, accumulate, ws, n, None),
        "wgrad": lambda: lib.moe_grouped_gemm_wgrad(g, ptr, ptr, pairs, off, ptr, dtype, accumulate, ws, n,
                                                    None),
        "int8": lambda: lib.moe_grouped_gemm_int8(g, ptr, ptr, pairs, off, ptr, ptr, ptr, dtype, ws, n, None),
    }


@pytest.mark.parametrize("change,status", [
    (dict(P=-1), 1), (dict(P=1 << 31), 1), (dict(S=-1), 1), (dict(S=1 << 31), 1), (dict(E=0), 1),
    (dict(k=0), 1), (dict(N=0), 1), (dict(N=12), 1), (dict(K=0), 1), (dict(K=12), 1),
    (dict(E=257), 2), (dict(N=65536 + 16), 2), (dict(K=65536 + 16), 2),
])
def test_shapes(lib, change, status):
    keep, good = _aligned()
    g = gemm(**change)
    for name, call in calls(lib, g, good).items():
        assert call() == status, (name, lib.moe_last_error())
        assert lib.moe_last_error()
    assert moe.moe_gemm_workspace_bytes(g) == 0


def test_int8_needs_multiples_of_sixteen(lib):
    keep, good = _aligned()
    assert calls(lib, gemm(K=24), good)["int8"]() == 1
    assert b"16" in lib.moe_last_error()
    assert lib.moe_quantize_rows_int8(4, 24, good, good, good, None) == 1
    assert lib.moe_quantize_rows_int8(-1, 32, good, good, good, None) == 1
    assert lib.moe_quantize_rows_int8(4, 65552, good, good, good, None) == 2
    assert lib.moe_quantize_rows_int8(4, 32, None, good, good, None) == 1
    assert lib.moe_quantize_rows_int8(0, 32, None, None, None, None) == 0


def test_pointers(lib):
    keep, good = _aligned()
    keep2, odd = _aligned(8)
    g = gemm()
    for name, call in calls(lib, g, None, off=good).items():
        assert call() == 1, name
    for name, call in calls(lib, g, odd).items():
        assert call() == 1, name
        assert b"aligned" in lib.moe_last_error()
    # offsets may be left out with one group only
    assert lib.moe_grouped_gemm(g, good, None, None, good, good, 0, None, 0, None) == 1
    # fewer rows than positions without sorted_pairs; no rows at all with them
    short = gemm(S=63)
    assert calls(lib, short, good)["gemm"]() == 1
    assert calls(lib, short, good)["wgrad"]() == 1
    assert calls(lib, short, good)["int8"]() == 1
    none = gemm(S=0, k=2)
    assert calls(lib, none, good, pairs=good)["gemm"]() == 1
    assert calls(lib, g, good, pairs=odd)["gemm"]() == 1


def test_output_types(lib):
    keep, good = _aligned()
    g = gemm()
    for name, call in calls(lib, g, good, dtype=7).items():
        assert call() == 1, name
    for name in ("dgrad", "wgrad"):
        assert calls(lib, g, good, dtype=1, accumulate=1)[name]() == 1
        assert b"fp32" in lib.moe_last_error()


def test_workspace(lib):
    keep, good = _aligned()
    keep2, odd = _aligned(8)
    g = gemm(P=4, S=4, E=1, K=16384, N=128)
    need = moe.moe_gemm_workspace_bytes(g)
    assert need > 0
    args = (good, None, good, good, good, 0)
    assert lib.moe_grouped_gemm(g, *args, None, need, None) == 3
    assert lib.moe_grouped_gemm(g, *args, good, need - 1, None) == 3
    assert lib.moe_grouped_gemm(g, *args, odd, need, None) == 3
    # one size for every call on the shape, and none for no positions
    assert moe.moe_gemm_workspace_bytes(gemm(P=0)) == 0


def test_workspace_stays_small():
    """The scratch of split reductions stays below 512 MiB over the range of
    shapes (reductions are split where there are few output tiles)."""
    rng = np.random.default_rng(0)
    for _ in range(3000):
        E = int(np.exp(rng.uniform(0, np.log(256.99))))
        N, K = (8 * int(np.exp(rng.uniform(np.log(1), np.log(8192)))) for _ in range(2))
        P = int(np.exp(rng.uniform(0, np.log(1 << 20))))
        g = moe.MoEGemmProblem(P, P, E, N, K, 1)
        assert moe.moe_gemm_workspace_bytes(g) <= 512 << 20, (P, E, N, K)


def test_no_positions(lib):
    g = gemm(P=0)
    keep, good = _aligned()
    assert lib.moe_grouped_gemm(g, None, None, None, None, None, 0, None, 0, None) == 0
    assert lib.moe_grouped_gemm_dgrad(g, None, None, None, None, 0, 0, None, 0, None) == 0
    assert lib.moe_grouped_gemm_int8(g, None, None, None, None, None, None, None, 0, None, 0, None) == 0
    # the weight gradient has an output all the same
    assert lib.moe_grouped_gemm_wgrad(g, None, None, None, good, None, 0, 0, None, 0, None) == 1


def test_expert_calls(lib):
    keep, good = _aligned()
    p = moe.MoEProblem(8, 256, 128, 16, 4, 2, 4, 1.0)
    n8, nb = moe.moe_int8_workspace_bytes(p), moe.moe_backward_workspace_bytes(p)
    assert n8 > 0 and nb > 0
    a8 = (good,) * 10
    assert lib.moe_expert_ffn_int8(p, *a8, None, n8, None) == 3
    assert lib.moe_expert_ffn_int8(p, *a8, good, n8 - 1, None) == 3
    assert lib.moe_expert_ffn_int8(p, *((None,) + a8[1:]), good, n8, None) == 1
    ab = (good,) * 11
    assert lib.moe_expert_ffn_backward(p, *ab, 0, 0, good, nb - 1, None) == 3
    assert lib.moe_expert_ffn_backward(p, *ab, 1, 1, good, nb, None) == 1
    assert lib.moe_expert_ffn_backward(p, *ab, 5, 0, good, nb, None) == 1
    for i in range(11):
        args = tuple(None if j == i else good for j in range(11))
        assert lib.moe_expert_ffn_backward(p, *args, 0, 0, good, nb, None) == 1, i
    fwd = (good, good, None) + (good,) * 7
    assert lib.moe_forward_int8(p, *fwd, 9, None, None, good, good, n8, None) == 1
    assert lib.moe_forward_int8(p, *fwd, 0, None, None, None, good, n8, None) == 1
    bad = moe.MoEProblem(8, 100, 128, 16, 4, 2, 4, 1.0)
    assert moe.moe_int8_workspace_bytes(bad) == 0 and moe.moe_backward_workspace_bytes(bad) == 0


def test_binding_checks(monkeypatch):
    """The binding refuses tensors of another type, device, size or layout
    before it calls the library."""
    monkeypatch.setattr(torch.cuda, "current_device", lambda: -1)  # the "device" of CPU tensors
    g = gemm()
    a = torch.zeros((64, 48), dtype=torch.bfloat16)
    w = torch.zeros((4, 32, 48), dtype=torch.bfloat16)
    off = torch.zeros(5, dtype=torch.int32)
    out = torch.zeros((64, 32))
    with pytest.raises(TypeError):
        moe.moe_grouped_gemm(g, a.float(), None, off, w, out)
    with pytest.raises(TypeError):
        moe.moe_grouped_gemm(g, a, None, off.long(), w, out)
    with pytest.raises(TypeError):
        moe.moe_grouped_gemm(g, a, None, off, w, out.half())
    with pytest.raises(ValueError):
        moe.moe_grouped_gemm(g, a[:63], None, off, w, out)
    with pytest.raises(ValueError):
        moe.moe_grouped_gemm(g, a, None, off[:4], w, out)
    with pytest.raises(ValueError):
        moe.moe_grouped_gemm(g, a, None, off, w.transpose(1, 2), out)
    with pytest.raises(ValueError):
        moe.moe_grouped_gemm(g, None, None, off, w, out)
    with pytest.raises(ValueError):
        moe.moe_grouped_gemm(g, a, None, None, w, out)
    with pytest.raises(ValueError):
        moe.moe_quantize_rows_int8(a.reshape(-1), torch.zeros(64 * 48, dtype=torch.int8), torch.zeros(64))

    class OtherStream:
        device = torch.device("cuda", 1)
        cuda_stream = 0
    with pytest.raises(ValueError):
        moe.moe_grouped_gemm(g, a, None, off, w, out, stream=OtherStream())
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    with pytest.raises(ValueError):
        moe.moe_grouped_gemm(g, a, None, off, w, out)
