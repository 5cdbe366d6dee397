"""The grouped products at the limits of their documented sizes: positions close
to 2^31.  The inputs are zeros but for a few rows, so the outputs of all other
rows are zeros; the values are small whole numbers, so every sum is exact."""
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


def ws_for(moe, g):
    return torch.full((max(16, moe.moe_gemm_workspace_bytes(g)),), 0xFF, dtype=torch.uint8, device="cuda")


def count_where(x, pred, rows=1 << 27):
    """How many values of x satisfy pred, a slice of rows at a time."""
    return sum(int(torch.count_nonzero(pred(x[i:i + rows]))) for i in range(0, len(x), rows))


@pytest.mark.parametrize("op", ["product", "input_grad", "weight_grad", "int8"])
@pytest.mark.parametrize("P", [(1 << 31) - 40000, (1 << 31) - 1])
def test_positions_near_the_limit(moe, P, op):
    """Two experts, the second with all rows but seven."""
    K = 16 if op == "int8" else 8
    N = 8
    print(f"[case] {op} P={P}", flush=True)
    rng = np.random.default_rng(P % 1000)
    at = np.unique(np.concatenate([[0, 6, 7, 8, 127, 128, P // 2, P - 65, P - 64, P - 2, P - 1],
                                   rng.integers(0, P, 40)]))
    at_gpu = torch.from_numpy(at).cuda()
    e = torch.from_numpy((at >= 7).astype(np.int64)).cuda()
    gen = torch.Generator(device="cuda").manual_seed(P % 1000)
    whole = torch.int8 if op == "int8" else torch.bfloat16

    def some(shape):
        return torch.randint(-4, 5, shape, generator=gen, device="cuda")

    def rows(width):
        """[P, width] zeros with a few rows of whole numbers, and these rows."""
        full, few = torch.zeros((P, width), dtype=whole, device="cuda"), some((len(at), width))
        full[at_gpu] = few.to(whole)
        return full, few.double()

    off = torch.tensor([0, 7, P], dtype=torch.int32, device="cuda")
    w = some((2, N, K))
    g = problem(P, P, 2, N, K, 1)
    ws = ws_for(moe, g)
    if op == "weight_grad":
        a, few_a = rows(K)
        dout, few_d = rows(N)
        dw = torch.full((2, N, K), float("nan"), device="cuda")
        moe.moe_grouped_gemm_wgrad(g, dout, a, None, off, dw, ws)
        torch.cuda.synchronize()
        ref = torch.stack([few_d[e == i].T @ few_a[e == i] for i in range(2)])
        assert torch.equal(dw.double(), ref)
        return
    if op == "input_grad":
        x, few = rows(N)
        out = torch.full((P, K), float("nan"), dtype=torch.bfloat16, device="cuda")
        moe.moe_grouped_gemm_dgrad(g, x, off, w.to(whole), out, ws)
        ref = torch.bmm(few[:, None, :], w.double()[e])[:, 0]
    else:
        x, few = rows(K)
        out = torch.full((P, N), float("nan"), dtype=torch.bfloat16, device="cuda")
        ref = torch.bmm(w.double()[e], few[:, :, None])[:, :, 0]
        if op == "int8":
            moe.moe_grouped_gemm_int8(g, x, torch.ones(P, device="cuda"), None, off, w.to(whole),
                                      torch.ones((2, N), device="cuda"), out, ws)
        else:
            moe.moe_grouped_gemm(g, x, None, off, w.to(whole), out, ws)
    torch.cuda.synchronize()
    ref = ref.float().to(torch.bfloat16)
    assert torch.equal(out[at_gpu], ref)
    assert count_where(out, torch.isnan) == 0
    assert count_where(out, lambda t: t != 0) == int(torch.count_nonzero(ref))


@pytest.mark.parametrize("rows,K", [((1 << 26) + 3, 16), ((1 << 24) + 1, 2064)])
def test_quantize_more_rows_than_one_launch_dimension(moe, rows, K):
    """More workgroups than fit along one dimension of a launch; 4099 rows over
    and over, so every row's codes are known from the 64-bit reference."""
    from test_gpu_grouped import quantize_ref
    print(f"[case] quantize {rows} x {K}", flush=True)
    gen = torch.Generator().manual_seed(K)
    few = torch.randn((4099, K), generator=gen) * torch.exp(3 * torch.randn((4099, 1), generator=gen))
    few = few.to(torch.bfloat16)
    rc, rs = (t.cuda() for t in quantize_ref(few))
    few = few.cuda()
    step = 4099 * 128
    x = torch.empty((rows, K), dtype=torch.bfloat16, device="cuda")
    for i in range(0, rows, step):
        n = min(step, rows - i)
        x[i:i + n] = few.repeat(128, 1)[:n]
    codes = torch.full((rows, K), 99, dtype=torch.int8, device="cuda")
    scales = torch.full((rows,), float("nan"), device="cuda")
    moe.moe_quantize_rows_int8(x, codes, scales)
    torch.cuda.synchronize()
    rc, rs = rc.repeat(128, 1), rs.repeat(128)
    for i in range(0, rows, step):
        n = min(step, rows - i)
        assert torch.equal(codes[i:i + n], rc[:n]) and torch.equal(scales[i:i + n], rs[:n]), i


def test_int8_experts_of_more_positions_than_one_launch_dimension(moe):
    """2^24 + 8 positions: the rows of h quantised by a workgroup each.  4096
    tokens over and over with the same experts, so the same y over and over."""
    base, k, E, H, I = 4096, 8, 8, 128, 64
    T = (1 << 21) + 1
    print(f"[case] int8 experts, {T} tokens", flush=True)
    gen = torch.Generator(device="cuda").manual_seed(1)
    x0 = torch.randn((base, H), generator=gen, device="cuda").to(torch.bfloat16)
    x = x0.repeat(T // base + 1, 1)[:T].contiguous()

    def weights(*shape):
        return (torch.randint(-127, 128, shape, generator=gen, dtype=torch.int8, device="cuda"),
                torch.rand(shape[:2], generator=gen, device="cuda") * 1e-3 + 1e-3)
    w = [t for shape in ((E, I, H), (E, I, H), (E, H, I)) for t in weights(*shape)]

    def run(x):
        """Every token goes to every expert: expert e's positions are the tokens in order."""
        n = len(x)
        p = moe.MoEProblem(n, H, I, E, 1, 1, k, 1.0)
        pairs = (torch.arange(n, device="cuda", dtype=torch.int32)[None, :] * k
                 + torch.arange(E, device="cuda", dtype=torch.int32)[:, None]).reshape(-1).contiguous()
        off = torch.arange(E + 1, device="cuda", dtype=torch.int32) * n
        ws = torch.empty((moe.moe_int8_workspace_bytes(p),), dtype=torch.uint8, device="cuda")
        y = torch.full((n * k, H), float("nan"), device="cuda")
        moe.moe_expert_ffn_int8(p, x, pairs, off, *w, y, ws)
        torch.cuda.synchronize()
        return y.view(E, n, H)
    few, many = run(x0), run(x)
    assert not bool(torch.isnan(few).any())
    for i in range(0, T, base):
        n = min(base, T - i)
        assert torch.equal(many[:, i:i + n], few[:, :n]), i


@pytest.mark.parametrize("op,T", [("combine", (1 << 26) + 5), ("residual", (1 << 24) + 5)])
def test_combine_of_more_tokens_than_one_launch_dimension(moe, op, T):
    """One expert a token, its row the token's own: the combine that ends the
    whole passes and sums the gradients of a token's pairs.  Every token's row
    repeats one of 4096."""
    base, H = 4096, 128
    print(f"[case] {op} T={T}", flush=True)
    gen = torch.Generator(device="cuda").manual_seed(T % 1000)
    y0 = torch.randn((base, H), generator=gen, device="cuda")
    w0 = torch.rand((base, 1), generator=gen, device="cuda")
    gain = torch.rand((H,), generator=gen, device="cuda")

    def run(y, w):
        n = len(y)
        p = moe.MoEProblem(n, H, 64, 4, 1, 1, 1, 2.5)
        rows = torch.arange(n, device="cuda", dtype=torch.int32)
        if op == "combine":
            out = torch.full((n, H), float("nan"), dtype=torch.bfloat16, device="cuda")
            moe.moe_combine(p, y, rows, w, out)
        else:
            out = torch.ones((n, H), device="cuda")
            moe.moe_combine_residual(p, y, rows, w, gain, 1e-6, 3, out)
        torch.cuda.synchronize()
        return out

    def many(t):
        x = torch.empty((T, *t.shape[1:]), device="cuda")
        x[: T // base * base].view(-1, *t.shape).copy_(t)
        x[T // base * base:] = t[: T % base]
        return x
    few = run(y0, w0)
    assert not bool(torch.isnan(few).any()) and bool((few != 1).any())
    out = run(many(y0), many(w0))
    whole = T // base * base
    for i in range(0, whole, base * 1024):
        part = out[i:min(i + base * 1024, whole)].view(-1, base, H)
        assert bool((part == few).all()), i
    assert torch.equal(out[whole:], few[: T - whole])


def test_route_of_more_tokens_than_one_launch_dimension(moe):
    """2^29 + 70 tokens: every one is routed as the same token of a small batch."""
    base, T, H, E = 16384, (1 << 29) + 70, 128, 4
    print(f"[case] route T={T}", flush=True)
    gen = torch.Generator(device="cuda").manual_seed(7)
    x0 = torch.randn((base, H), generator=gen, device="cuda").to(torch.bfloat16)
    wr = torch.randn((E, H), generator=gen, device="cuda").to(torch.bfloat16)
    bias = torch.randn((E,), generator=gen, device="cuda")

    def run(x):
        p = moe.MoEProblem(len(x), H, 64, E, 1, 1, 1, 1.0)
        ids = torch.full((len(x),), -1, dtype=torch.int32, device="cuda")
        w = torch.full((len(x),), float("nan"), device="cuda")
        moe.moe_route(p, x, wr, bias, ids, w)
        torch.cuda.synchronize()
        return ids, w
    few = run(x0)
    assert len(few[0].unique()) > 1
    x = torch.empty((T, H), dtype=torch.bfloat16, device="cuda")
    whole = T // base * base
    x[:whole].view(-1, base, H).copy_(x0)
    x[whole:] = x0[: T - whole]
    many = run(x)
    for a, b in zip(many, few):
        assert bool((a[:whole].view(-1, base) == b).all()) and torch.equal(a[whole:], b[: T - whole])
