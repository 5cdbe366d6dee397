"""Products and gate_up on FP8 operands whose scales lie at the ends of the
range that moe_fp8.h allows: every product is a whole number of one unit, so
sums are exact wherever nothing is lost."""
import pytest
import torch

import _fp8block as f8

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    from group_limited_routing_router_amd import moe as m
    m.load_library()
    return m


def codes(gen, unit, most, *shape):
    """Whole numbers up to `most` times unit (those of 4 significant bits)."""
    v = torch.tensor([i for i in range(-most, most + 1) if f8.to_e4m3(torch.tensor(float(abs(i)))) == abs(i)])
    return f8.code_of(v[torch.randint(0, len(v), shape, generator=gen)].double() * unit)


TINY = 2.0 ** -9  # the smallest code

# scale bytes and units of the two operands; dequantised values below 2^127
ENDS = [(1, 250, TINY, 1.0), (250, 1, 1.0, TINY), (1, 254, 1.0, TINY), (254, 1, TINY, 1.0), (2, 246, TINY, 16.0),
        (246, 2, 16.0, TINY)]


@pytest.mark.parametrize("op", ["product", "input_grad"])
@pytest.mark.parametrize("ends", ENDS, ids=str)
def test_products(moe, ends, op):
    print(f"[case] {op} {ends}", flush=True)
    by, bx, uy, ux = ends
    P, N, K = 70, 160, 272
    gen = torch.Generator().manual_seed(1)
    red, cols = (K, N) if op == "product" else (N, K)
    # values of at most 7 or 224: below 2^127 on scales of up to 2^119 or 2^124
    y, w = codes(gen, uy, 7, P, red), codes(gen, ux, 7, 1, N, K)
    sy = torch.full((P, f8.pitch(red)), by, dtype=torch.uint8)
    sw = torch.full((1, f8.blocks(N), f8.blocks(K)), bx, dtype=torch.uint8)
    g = moe.MoEGemmProblem(P, P, 1, N, K, 1)
    ws = torch.full((max(16, moe.moe_gemm_workspace_bytes(g)),), 0xFF, dtype=torch.uint8, device="cuda")
    out = torch.full((P, cols), float("nan"), device="cuda")
    if op == "product":
        moe.moe_grouped_gemm_fp8_block(g, y.cuda(), sy.cuda(), None, None, w.cuda(), sw.cuda(), out, ws)
    else:
        moe.moe_grouped_gemm_fp8_block_dgrad(g, y.cuda(), sy.cuda(), None, w.cuda(), sw.cuda(), out, ws)
    wv, yv = f8.value_weights(w, sw)[0], f8.value_rows(y, sy)
    assert max(float(wv.abs().max()), float(yv.abs().max())) < 2.0 ** 127
    assert torch.equal(out.cpu().double(), yv @ (wv.T if op == "product" else wv))


# gate_up's: the lowest and the highest byte of either operand, beside one that
# brings gates to a few units or hundreds
GATED = [(3, 249, TINY, 1.0), (249, 3, 1.0, TINY), (3, 246, TINY, 16.0), (246, 3, 16.0, TINY), (4, 248, TINY, 1.0),
         (19, 234, TINY, 1.0), (254, 3, TINY, 1.0), (3, 254, 1.0, TINY)]


@pytest.mark.parametrize("T", [1, 24, 25, 100])
@pytest.mark.parametrize("ends", GATED, ids=str)
def test_gate_up(moe, ends, T):
    """h within half a step of its code beside 20 half steps of fp32 for the
    activation, on rows multiplied as bf16 (up to 24) and by the scaled
    instruction."""
    print(f"[case] gate_up {T} {ends}", flush=True)
    by, bx, uy, ux = ends
    H, I = 256, 128
    gen = torch.Generator().manual_seed(T)
    x = codes(gen, uy, 7, T, H)
    w = codes(gen, ux, 7, 2, I, H)
    sx = torch.full((T, f8.pitch(H)), by, dtype=torch.uint8)
    sw = torch.full((1, f8.blocks(I), f8.blocks(H)), bx, dtype=torch.uint8)
    p = moe.MoEProblem(T, H, I, 1, 1, 1, 1, 1.0)
    h = torch.full((T, I), 0x55, dtype=torch.uint8, device="cuda")
    hs = torch.full((T, f8.pitch(I)), 0x55, dtype=torch.uint8, device="cuda")
    moe.moe_expert_gate_up_fp8_block(p, x.cuda(), sx.cuda(), None, None, w[0].cuda(), sw.cuda(), w[1].cuda(), sw.cuda(),
                                     h, hs)
    xv = f8.value_rows(x, sx)
    g, u = (xv @ f8.value_weights(w[i:i + 1], sw)[0].T for i in (0, 1))
    ref = g / (1 + torch.exp(-g)) * u
    got = f8.value_rows(h.cpu(), hs.cpu())
    off = 20 * 2.0 ** -24 * ref.abs()
    top = (ref.abs() + off).amax(1, keepdim=True)
    assert float(top.min()) > 2.0 ** -90  # blocks below 2^-100 are zeros
    tol = 2.0 ** -4 * (ref.abs() + off) + 2.0 ** -10 * torch.exp2(f8.scale_exponents(top)[0]) + off
    assert float(((got - ref).abs() / tol).nan_to_num(nan=float("inf")).max()) <= 1.0
