"""Activations of more than 4 GiB, past the 32-bit offsets of the tiles that
gather rows."""
import numpy as np
import pytest
import torch

from _grouped import problem

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    from group_limited_routing_router_amd import moe as m
    m.load_library()
    yield m
    torch.cuda.empty_cache()


def test_token_gradients_of_many_tokens(moe):
    """The tokens' gradients gather nothing, so they are the same to the last
    bit whether the tokens fill 10 MB or more than 4 GiB.  One value in every
    row of x and dy, so g, u and dh are the same however they are summed; the
    sums over I that give dx are not."""
    T, few, H, I, E = 420_000, 1000, 5120, 64, 4
    print(f"[case] {T} tokens", flush=True)
    gen = torch.Generator(device="cuda").manual_seed(3)

    def one_hot(at):
        t = torch.zeros((T, H), dtype=torch.bfloat16, device="cuda")
        t[torch.arange(T, device="cuda"), at] = 1
        return t
    x, dy = (one_hot(torch.randint(0, H, (T,), generator=gen, device="cuda")) for _ in range(2))
    w = [torch.randn(s, generator=gen, device="cuda").to(torch.bfloat16)
         for s in ((E, I, H), (E, I, H), (E, H, I))]

    def run(n, counts):
        p = moe.MoEProblem(n, H, I, E, 1, 1, 1, 1.0)
        off = torch.from_numpy(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)).cuda()
        pairs = torch.arange(n, dtype=torch.int32, device="cuda")
        ws = torch.full((moe.moe_backward_workspace_bytes(p),), 0xFF, dtype=torch.uint8, device="cuda")
        dx = torch.full((n, H), float("nan"), device="cuda")
        dw = [torch.empty_like(t) for t in w]
        moe.moe_expert_ffn_backward(p, x[:n], pairs, off, *w, dy[:n], dx, *dw, ws)
        torch.cuda.synchronize()
        return dx
    small = run(few, [few, 0, 0, 0])
    large = run(T, [T // 4] * 4)
    assert bool(torch.isfinite(large).all()) and bool((small != 0).any())
    assert torch.equal(large[:few], small)


def test_int8_rows_past_four_gigabytes(moe):
    """The int8 product of rows gathered from 4.3 GB of codes, bit for bit."""
    S, K, N, P, k = 840_000, 5120, 72, 96, 2
    print(f"[case] int8 gather from {S} x {K}", flush=True)
    gen = torch.Generator(device="cuda").manual_seed(1)
    at = np.linspace(0, S - 1, P).astype(np.int64)[::-1].copy()
    rows = torch.from_numpy(at).cuda()
    a = torch.zeros((S, K), dtype=torch.int8, device="cuda")
    a[rows] = torch.randint(-128, 128, (P, K), generator=gen, dtype=torch.int8, device="cuda")
    a_scale = torch.full((S,), float("nan"), device="cuda")
    a_scale[rows] = torch.rand((P,), generator=gen, device="cuda") + 0.01
    w = torch.randint(-128, 128, (3, N, K), generator=gen, dtype=torch.int8, device="cuda")
    w_scale = torch.rand((3, N), generator=gen, device="cuda") + 0.01
    spans = ((0, 3, 20), (2, 20, P - 5))      # expert 1 idle, rows of no expert at both ends
    off = torch.tensor([3, 20, 20, P - 5], dtype=torch.int32, device="cuda")
    pairs = torch.from_numpy((at * k + np.arange(P) % k).astype(np.int32)).cuda()
    g = problem(P, S, 3, N, K, k)
    ws = torch.empty((max(16, moe.moe_gemm_workspace_bytes(g)),), dtype=torch.uint8, device="cuda")
    for dtype in (torch.float32, torch.bfloat16):
        out = torch.full((P, N), float("nan"), dtype=dtype, device="cuda")
        moe.moe_grouped_gemm_int8(g, a, a_scale, pairs, off, w, w_scale, out, ws)
        torch.cuda.synchronize()
        for e, i, j in spans:
            acc = a[rows[i:j]].double() @ w[e].double().T
            ref = acc.float() * (a_scale[rows[i:j]][:, None] * w_scale[e][None, :])
            assert torch.equal(out[i:j], ref.to(dtype)), e
        assert bool(torch.isnan(out[:3].float()).all()) and bool(torch.isnan(out[P - 5:].float()).all())
