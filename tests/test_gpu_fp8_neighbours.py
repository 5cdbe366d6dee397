"""What stands beside the FP8 products: calls on bf16 operands need no more
workspace than their own sums, and the norm's gradient may overwrite x."""
import pytest
import torch

from _grouped import offsets_of

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def moe():
    from group_limited_routing_router_amd import moe as m
    m.load_library()
    return m


def test_workspace_of_bf16_gradients(moe):
    """Its sums are those of two parts: the same product splits in four in FP8."""
    P, H, I = 4, 2816, 8128  # P I in whole units of 256 bytes
    p = moe.MoEProblem(1, H, I, 77, 1, 1, P, 1.0)
    assert moe.moe_backward_workspace_bytes(p) == 3 * P * I * 4 + 3 * P * I * 2 + 2 * P * H * 4


@pytest.mark.gpu
def test_bf16_products_without_workspace(moe):
    """A shape whose reduction is split in FP8 and not in bf16: the calls on bf16
    go without a workspace, and give what they give with one."""
    P, E, N, K = 2191, 8, 13744, 1216
    gen = torch.Generator(device="cuda").manual_seed(5)
    counts = torch.bincount(torch.randint(0, E, (P,), generator=gen, device="cuda"), minlength=E)
    off = offsets_of(counts.cpu().numpy()).cuda()
    g = moe.MoEGemmProblem(P, P, E, N, K, 1)
    need = moe.moe_gemm_workspace_bytes(g)
    assert need > 0
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")
    a = torch.randn((P, K), generator=gen, device="cuda").to(BF16)
    w = torch.randn((E, N, K), generator=gen, device="cuda").to(BF16)
    dout = torch.randn((P, N), generator=gen, device="cuda").to(BF16)
    for call, shape in ((lambda o, s: moe.moe_grouped_gemm(g, a, None, off, w, o, s), (P, N)),
                        (lambda o, s: moe.moe_grouped_gemm_dgrad(g, dout, off, w, o, s), (P, K)),
                        (lambda o, s: moe.moe_grouped_gemm_wgrad(g, dout, a, None, off, o, s), (E, N, K))):
        out = [torch.full(shape, float("nan"), dtype=BF16, device="cuda") for _ in range(2)]
        call(out[0], None)
        call(out[1], ws)
        assert torch.equal(out[0].view(torch.int16), out[1].view(torch.int16))
        assert not out[0].isnan().any()


@pytest.mark.gpu
@pytest.mark.parametrize("center", [False, True])
@pytest.mark.parametrize("rows,H", [(700, 256), (700, 5120), (300, 16384)])
def test_norm_gradient_over_x(moe, rows, H, center):
    gen = torch.Generator(device="cuda").manual_seed(6)
    x = torch.randn((rows, H), generator=gen, device="cuda")
    dy = torch.randn((rows, H), generator=gen, device="cuda").to(BF16)
    w = torch.randn((H,), generator=gen, device="cuda")
    y, stats = torch.empty_like(x), torch.empty((rows, 2), device="cuda")
    moe.moe_norm(x, w, None, 1e-6, y, stats, center=center)
    ws = torch.empty((moe.moe_norm_workspace_bytes(rows, H),), dtype=torch.uint8, device="cuda")
    got = []
    for over in (False, True):
        xs, dw, db = x.clone(), torch.empty_like(w), torch.empty_like(w)
        dx = xs if over else torch.empty_like(x)
        moe.moe_norm_backward(dy, xs, w, stats, dx, dw, db, ws, center=center)
        got.append((dx, dw, db))
    for a, b in zip(*got):
        assert torch.equal(a, b)
