"""h of the int8 experts: its codes to the nearest, ties to even, and silu over
the whole range of gates.  The down projection picks out single values of h, so
y holds their codes times the row's scale."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    from group_limited_routing_router_amd import moe as m
    m.load_library()
    return m


def expert(moe, x, w_gate, s_gate, w_up, s_up, I):
    """y of one expert that takes every row, w_down[m, n] = 1 where m = n (the
    first I columns of y are h's codes times the row's scale)."""
    T, H = x.shape
    p = moe.MoEProblem(T, H, I, 1, 1, 1, 1, 1.0)
    pairs = torch.arange(T, dtype=torch.int32, device="cuda")
    off = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    w_down = torch.zeros((1, H, I), dtype=torch.int8, device="cuda")
    n = torch.arange(min(H, I), device="cuda")
    w_down[0, n, n] = 1
    y = torch.full((T, H), float("nan"), device="cuda")
    ws = torch.full((moe.moe_int8_workspace_bytes(p),), 0xFF, dtype=torch.uint8, device="cuda")
    moe.moe_expert_ffn_int8(p, x, pairs, off, w_gate, s_gate, w_up, s_up, w_down,
                            torch.ones((1, H), device="cuda"), y, ws)
    torch.cuda.synchronize()
    return y[:, :I]


@pytest.mark.parametrize("I", [64, 128])
def test_ties_of_h(moe, I):
    """Every value of a row is half its largest one: 63.5, to even 64.  The
    gates are equal along the row and the up scales differ by a factor of two,
    so the halves are exact."""
    T, H = 4096, 128
    print(f"[case] ties I={I}", flush=True)
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.zeros((T, H), dtype=torch.bfloat16, device="cuda")
    x[:, 0] = torch.exp(torch.randn((T,), generator=gen, device="cuda")).to(torch.bfloat16)
    w = torch.zeros((1, I, H), dtype=torch.int8, device="cuda")
    w[..., 0] = 91
    s_gate = torch.full((1, I), 0.0137, device="cuda")
    s_up = torch.full((1, I), 0.00731, device="cuda")
    s_up[0, 1:] /= 2
    s_up[0, 2::2] *= -1
    y = expert(moe, x, w, s_gate, w, s_up, I).double()
    codes = torch.round(127 * y / y[:, :1])
    want = torch.full((I,), 64.0, dtype=torch.float64, device="cuda")
    want[0], want[2::2] = 127, -64
    assert torch.equal(codes, want.expand(T, I))
