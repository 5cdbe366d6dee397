"""The FP8 experts' gradients where every sum of the pass is exact, so that the
roundings of the definition are the only ones left (_fp8exact.py): on every tile
of the two-matrix product dx = [dg | du] . [gate; up], split and not, with
weights past the caches and not, with more stages than the scales held in
registers; on every tile of the gated pass, gathered and not."""
import pytest
import torch

from _fp8exact import BF16, F32, NAMES, WholeExperts, gradients, off_by
from _fp8plan import plan

# (T, k, E, H, I): the tile, weights past the caches and parts of the two-matrix
# product; the same of the gated pass
SHAPES = {
    (1, 1, 1, 128, 64): ((32, False, 1), (32, False, 1)),
    (24, 1, 1, 256, 704): ((32, False, 1), (32, False, 1)),
    (118, 1, 2, 1792, 2624): ((32, False, 1), (128, False, 1)),     # 42 stages
    (1, 1, 1, 256, 10432): ((32, False, 16), (32, False, 1)),       # parts that start inside a word of scales
    (120, 2, 2, 384, 4160): ((32, False, 8), (128, False, 1)),
    (1024, 1, 256, 512, 1088): ((32, True, 1), (32, True, 1)),
    (41, 2, 64, 1280, 1984): ((32, True, 2), (32, True, 1)),
    (16, 1, 16, 1536, 5440): ((32, True, 1), (32, False, 1)),       # 86 stages
    (70, 1, 1, 256, 704): ((32, False, 1), (128, False, 1)),
    (901, 2, 8, 1152, 704): ((128, False, 1), (128, False, 1)),
    (732, 2, 2, 1408, 2624): ((128, False, 1), (128, False, 1)),    # 42 stages
    (811, 1, 1, 1280, 3136): ((128, False, 2), (128, False, 1)),
    (448, 2, 2, 1152, 5248): ((128, False, 2), (128, False, 1)),    # 41 stages a part
    (7168, 1, 256, 512, 1088): ((128, True, 1), (128, True, 1)),
    (916, 2, 64, 1152, 2304): ((128, True, 2), (128, True, 1)),
    (6000, 2, 3, 1024, 1344): ((256, False, 1), (256, False, 1)),
    (2000, 2, 2, 2048, 2624): ((256, False, 1), (256, False, 1)),   # 42 stages
    (3355, 1, 1, 1280, 4800): ((256, False, 2), (256, False, 1)),
}

# (T, H, I) of dense layers without a dispatch
DENSE = [(1, 256, 704), (9, 384, 320), (24, 256, 704), (3, 8192, 18432), (25, 256, 704), (70, 640, 192),
         (30, 8192, 18432), (2100, 640, 4160)]


def tiles_of(T, k, E, H, I):
    return plan("pair", T * k, E, I, H), plan("gated", T * k, E, I, H)


@pytest.fixture(scope="module")
def moe():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    from group_limited_routing_router_amd import moe as m
    m.load_library()
    yield m
    torch.cuda.empty_cache()


def workspace(n):
    return torch.full((max(16, n),), 0xFF, dtype=torch.uint8, device="cuda")


def backward(moe, c, dx_dtype, dw_dtype, dispatch=True):
    p = c.problem()
    dx = torch.full((c.P, c.H), float("nan"), dtype=dx_dtype, device="cuda")
    dw = [torch.full(c.q[n].shape, float("nan"), dtype=dw_dtype, device="cuda") for n in NAMES]
    where = (c.pairs, c.offsets) if dispatch else (None, None)
    moe.moe_expert_ffn_fp8_block_backward(p, c.x, *where, *c.weights(), c.dy, dx, *dw,
                                          workspace(moe.moe_fp8_block_backward_workspace_bytes(p)))
    torch.cuda.synchronize()
    return [dx, *dw]


@pytest.mark.gpu
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_gradients(moe, shape):
    print(f"[case] exact {shape}", flush=True)
    assert tiles_of(*shape) == SHAPES[shape]
    c = WholeExperts(*shape, seed=sum(shape), device="cuda")
    want = gradients(c)
    for dx_dtype, dw_dtype in ((F32, F32), (BF16, BF16)):
        got = backward(moe, c, dx_dtype, dw_dtype)
        worst = [off_by(g, r, t, d) for g, (r, t), d in zip(got, want, (dx_dtype, dw_dtype, dw_dtype, dw_dtype))]
        print("   ", worst, flush=True)
        assert max(worst) <= 1.0


def forward(moe, c, dispatch):
    p = c.problem()
    y = torch.full((c.P, c.H), float("nan"), device="cuda")
    where = (c.pairs, c.offsets) if dispatch else (None, None)
    moe.moe_expert_ffn_fp8_block(p, c.x, *where, *c.weights(), y, workspace(moe.moe_fp8_block_workspace_bytes(p)))
    torch.cuda.synchronize()
    return y


@pytest.mark.gpu
@pytest.mark.parametrize("T,H,I", DENSE)
def test_dense_layer_without_dispatch(moe, T, H, I):
    """The same, to the bit, as with the dispatch written out, which the tests
    above hold to the definition; small ones are held to it themselves."""
    print(f"[case] dense {T} {H} {I}", flush=True)
    c = WholeExperts(T, 1, 1, H, I, seed=T, device="cuda", order=True)
    assert torch.equal(forward(moe, c, False), forward(moe, c, True))
    for got, want in zip(backward(moe, c, F32, F32, False), backward(moe, c, F32, F32, True)):
        assert torch.equal(got, want) and not got.isnan().any()
    if H * I < 4e6:
        got = backward(moe, c, F32, F32, False)
        assert max(off_by(g, r, t, F32) for g, (r, t) in zip(got, gradients(c))) <= 1.0
