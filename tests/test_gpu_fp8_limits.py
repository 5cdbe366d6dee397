"""FP8 by blocks and the norm at the edges of their ranges: every tile, split and
weight stream, operands and outputs past 4 GiB, calls captured into graphs, the
binding's refusals."""
import pytest
import torch

import _fp8block as f8
from _grouped import offsets_of

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
NAN = float("nan")


@pytest.fixture(scope="module")
def moe():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    from group_limited_routing_router_amd import moe as m
    m.load_library()
    return m


def whole(gen, *shape):
    """Codes of the whole numbers -8 .. 8, drawn on the GPU."""
    v = torch.arange(-8, 9, device="cuda").float().to(torch.float8_e4m3fn).view(torch.uint8)
    return v[torch.randint(0, 17, shape, generator=gen, device="cuda")]


def scales(gen, *shape):
    return torch.randint(126, 129, shape, generator=gen, device="cuda", dtype=torch.uint8)


def spans(off):
    o = off.tolist()
    return [(e, o[e], o[e + 1]) for e in range(len(o) - 1) if o[e + 1] > o[e]]


def draw_counts(gen, P, E):
    c = torch.bincount(torch.randint(0, E, (P,), generator=gen, device="cuda"), minlength=E)
    return c.cpu().numpy()


def workspace(n):
    return torch.full((max(16, n),), 0xFF, dtype=torch.uint8, device="cuda")


@pytest.mark.parametrize("op", ["product", "input_grad"])
@pytest.mark.parametrize("shape", [
    (6000, 3, 2064, 1040),     # 256-row tiles, ragged
    (9000, 2, 1040, 5264),     # and a reduction past one load of scales
    (1000, 256, 1040, 1024),   # a weight stream and few rows
    (8000, 256, 1040, 1024),   # and more
    (9, 1, 256, 16384),        # split sums
    (30, 1, 512, 20480),
    (2, 1, 20480, 256),
    (500, 5, 2560, 784),
], ids=lambda s: "x".join(map(str, s)))
def test_tiles(moe, op, shape):
    """Sums of whole numbers come out exactly, on every tile and split."""
    print(f"[case] tiles {op} {shape}", flush=True)
    P, E, N, K = shape
    gen = torch.Generator(device="cuda").manual_seed(P + K)
    off = offsets_of(draw_counts(gen, P, E)).cuda()
    down = op == "input_grad"
    red, cols = (N, K) if down else (K, N)
    a, sa = whole(gen, P, red), scales(gen, P, f8.pitch(red))
    w, sw = whole(gen, E, N, K), scales(gen, E, f8.blocks(N), f8.blocks(K))
    g = moe.MoEGemmProblem(P, P, E, N, K, 1)
    ws = workspace(moe.moe_gemm_workspace_bytes(g))
    out = torch.full((P, cols), NAN, device="cuda")
    if down:
        moe.moe_grouped_gemm_fp8_block_dgrad(g, a, sa, off, w, sw, out, ws)
    else:
        moe.moe_grouped_gemm_fp8_block(g, a, sa, None, off, w, sw, out, ws)
    torch.cuda.synchronize()
    for e, i, j in spans(off):
        x = f8.value_weights(w[e:e + 1], sw[e:e + 1])[0]
        x = x if down else x.T
        y = f8.value_rows(a[i:j], sa[i:j])
        # every term is a whole number of quarters, and so is every sum of them
        assert float((y.abs() @ x.abs()).max()) * 4 < 2 ** 24, "not exact in fp32"
        assert torch.equal(out[i:j].double(), y @ x), e


def gated(moe, gen, P, E, H, I, x, sx, off, w, pairs=None):
    p = moe.MoEProblem(P, H, I, E, 1, 1, 1, 1.0)
    h = torch.full((P, I), 0x55, dtype=torch.uint8, device="cuda")
    hs = torch.full((P, f8.pitch(I)), 0x55, dtype=torch.uint8, device="cuda")
    pairs = torch.arange(P, dtype=torch.int32, device="cuda") if pairs is None else pairs
    moe.moe_expert_gate_up_fp8_block(p, x, sx, pairs, off, *w, h, hs)
    torch.cuda.synchronize()
    return h, hs


@pytest.mark.parametrize("P,E,H,I", [
    (1000, 256, 1024, 640),   # 32 rows, weights past the caches
    (7000, 256, 1024, 640),   # 128 rows, past the caches
    (4000, 256, 640, 320),    # 32 rows
    (12000, 24, 640, 1472),   # 256 rows
    (3000, 20, 384, 192),     # 128 rows, few tiles
])
def test_gated_tiles(moe, P, E, H, I):
    """g and u are exact sums of whole numbers (scaled down to gates of a few
    units), so h is off by the activation and its own rounding alone."""
    print(f"[case] gated tiles {P} {E} {H} {I}", flush=True)
    gen = torch.Generator(device="cuda").manual_seed(P)
    off = offsets_of(draw_counts(gen, P, E)).cuda()
    x, sx = whole(gen, P, H), torch.full((P, f8.pitch(H)), 117, dtype=torch.uint8, device="cuda")
    w = []
    for _ in range(2):
        w += [whole(gen, E, I, H), scales(gen, E, f8.blocks(I), f8.blocks(H))]
    h, hs = gated(moe, gen, P, E, H, I, x, sx, off, w)
    got = f8.value_rows(h, hs)
    xv = f8.value_rows(x, sx)
    for e, i, j in spans(off):
        g = xv[i:j] @ f8.value_weights(w[0][e:e + 1], w[1][e:e + 1])[0].T
        u = xv[i:j] @ f8.value_weights(w[2][e:e + 1], w[3][e:e + 1])[0].T
        ref = g / (1 + torch.exp(-g)) * u
        off_by = 20 * 2.0 ** -24 * ref.abs()
        top = torch.nn.functional.pad(ref.abs() + off_by, (0, -I % 128)).reshape(j - i, -1, 128).amax(2)
        scale = torch.exp2(f8.scale_exponents(top)[0]).repeat_interleave(128, 1)[:, :I]
        tol = 2.0 ** -4 * (ref.abs() + off_by) + 2.0 ** -10 * scale + off_by
        assert float(((got[i:j] - ref).abs() / tol).max()) <= 1.0, e


def test_operands_past_four_gib(moe):
    """Rows of y, weights and outputs whose bytes pass 32 bits."""
    gen = torch.Generator(device="cuda").manual_seed(1)
    P, R = 290_000, 16384  # 4.75 GB of codes
    a = whole(gen, 1000, R).repeat(P // 1000, 1)
    sa = torch.full((P, f8.pitch(R)), 126, dtype=torch.uint8, device="cuda")
    off = torch.tensor([0, 5, P - 300, P], dtype=torch.int32, device="cuda")
    for down in (False, True):
        N, K = (R, 32) if down else (32, R)
        w, sw = whole(gen, 3, N, K), scales(gen, 3, f8.blocks(N), f8.blocks(K))
        g = moe.MoEGemmProblem(P, P, 3, N, K, 1)
        out = torch.full((P, 32), NAN, device="cuda")
        ws = workspace(moe.moe_gemm_workspace_bytes(g))
        if down:
            moe.moe_grouped_gemm_fp8_block_dgrad(g, a, sa, off, w, sw, out, ws)
        else:
            moe.moe_grouped_gemm_fp8_block(g, a, sa, None, off, w, sw, out, ws)
        torch.cuda.synchronize()
        for e, i, j in ((0, 0, 5), (1, 5, 300), (1, P - 600, P - 300), (2, P - 300, P)):
            x = f8.value_weights(w[e:e + 1], sw[e:e + 1])[0]
            ref = f8.value_rows(a[i:j], sa[i:j]) @ (x if down else x.T)
            assert torch.equal(out[i:j].double(), ref), (down, i)
        assert torch.isfinite(out).all()
        del out, w, ws
    # rows of bf16 past 4 GiB to codes
    del a, sa
    torch.cuda.empty_cache()
    x = torch.randn((300, 5120), generator=gen, device="cuda").to(BF16).repeat(1700, 1)
    codes, s = torch.empty(x.shape, dtype=torch.uint8, device="cuda"), torch.empty((len(x), 40), dtype=torch.uint8, device="cuda")
    moe.moe_quantize_rows_fp8_block(x, codes, s)
    torch.cuda.synchronize()
    want, ws = f8.quantise_rows(x[:300])
    for i in (0, 300 * 1000, len(x) - 300):
        assert torch.equal(codes[i:i + 300], want) and torch.equal(s[i:i + 300], ws)


def test_wide_output(moe):
    """[P,N] of 4.8 GB, two experts."""
    gen = torch.Generator(device="cuda").manual_seed(2)
    P, N, K = 40_000, 60_000, 32
    a, sa = whole(gen, P, K), scales(gen, P, 4)
    w, sw = whole(gen, 2, N, K), scales(gen, 2, f8.blocks(N), 1)
    off = torch.tensor([0, 100, P], dtype=torch.int32, device="cuda")
    g = moe.MoEGemmProblem(P, P, 2, N, K, 1)
    out = torch.full((P, N), NAN, dtype=BF16, device="cuda")
    moe.moe_grouped_gemm_fp8_block(g, a, sa, None, off, w, sw, out, workspace(moe.moe_gemm_workspace_bytes(g)))
    torch.cuda.synchronize()
    for e, i, j in ((0, 0, 100), (1, 100, 300), (1, P - 200, P)):
        ref = f8.value_rows(a[i:j], sa[i:j]) @ f8.value_weights(w[e:e + 1], sw[e:e + 1])[0].T
        assert torch.equal(out[i:j], ref.float().to(BF16))


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_norm_past_four_gib(moe, dtype):
    gen = torch.Generator(device="cuda").manual_seed(3)
    rows, H = (140_000, 8192) if dtype == F32 else (290_000, 8192)
    few = torch.randn((1000, H), generator=gen, device="cuda").to(dtype)
    x = few.repeat(rows // 1000, 1)
    w = 1 + 0.1 * torch.randn((H,), generator=gen, device="cuda")
    out, stats = torch.empty(x.shape, dtype=BF16, device="cuda"), torch.empty((rows, 2), device="cuda")
    moe.moe_norm(x, w, None, 1e-6, out, stats, center=True)
    one, s1 = torch.empty((1000, H), dtype=BF16, device="cuda"), torch.empty((1000, 2), device="cuda")
    moe.moe_norm(few, w, None, 1e-6, one, s1, center=True)
    dx = torch.empty_like(x)
    dw, db = torch.empty(H, device="cuda"), torch.empty(H, device="cuda")
    moe.moe_norm_backward(out, x, w, stats, dx, dw, db, workspace(moe.moe_norm_workspace_bytes(rows, H)), center=True)
    d1, w1, b1 = torch.empty_like(few), torch.empty(H, device="cuda"), torch.empty(H, device="cuda")
    moe.moe_norm_backward(one, few, w, s1, d1, w1, b1, workspace(moe.moe_norm_workspace_bytes(1000, H)), center=True)
    torch.cuda.synchronize()
    for i in (0, rows - 1000):
        assert torch.equal(out[i:i + 1000], one) and torch.equal(stats[i:i + 1000], s1) and torch.equal(dx[i:i + 1000], d1)
    # the columns' sums: rows / 1000 times those of the few, each side off by
    # its own additions: at most (rows / 256 + 600) 2^-24 of the magnitudes
    n = rows // 1000
    xh = (few.double() - s1[:, :1].double()) * s1[:, 1:].double()
    for got, part, mag in ((dw, w1, (one.double() * xh).abs().sum(0)), (db, b1, one.double().abs().sum(0))):
        tol = n * mag * (rows / 256 + 1800) * 2.0 ** -24
        assert float(((got.double() - n * part.double()).abs() / tol).max()) <= 1.0


def test_graph_of_products(moe):
    """Quantisation and split products captured, replayed on other rows, with
    eager calls between."""
    gen = torch.Generator(device="cuda").manual_seed(4)
    P, N, K = 20, 512, 8192
    g = moe.MoEGemmProblem(P, P, 1, N, K, 1)
    w = (0.05 * torch.randn((1, N, K), generator=gen, device="cuda")).to(BF16)
    wq = torch.empty(w.shape, dtype=torch.float8_e4m3fn, device="cuda")
    sw = torch.empty((1, f8.blocks(N), f8.blocks(K)), dtype=torch.uint8, device="cuda")
    moe.moe_quantize_weights_fp8_block(w, wq, sw)
    x = torch.randn((P, K), generator=gen, device="cuda").to(BF16)
    xq, sx = torch.empty(x.shape, dtype=torch.float8_e4m3fn, device="cuda"), torch.empty((P, f8.pitch(K)), dtype=torch.uint8, device="cuda")
    out, ws = torch.empty((P, N), device="cuda"), workspace(moe.moe_gemm_workspace_bytes(g))
    assert moe.moe_gemm_workspace_bytes(g) > 0

    def step():
        moe.moe_quantize_rows_fp8_block(x, xq, sx)
        moe.moe_grouped_gemm_fp8_block(g, xq, sx, None, None, wq, sw, out, ws)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(4):
        x.copy_(torch.randn((P, K), generator=gen, device="cuda") * 2.0 ** i)
        step()
        want = out.clone()
        out.fill_(NAN)
        ws.fill_(0xFF)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_binding_refuses(moe):
    g = moe.MoEGemmProblem(32, 32, 2, 32, 48, 1)
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8, device="cuda")  # noqa: E731
    off = torch.zeros(3, dtype=torch.int32, device="cuda")
    good = [u8(32, 48), u8(32, 4), None, off, u8(2, 32, 48), u8(2, 1, 1), torch.zeros((32, 32), device="cuda")]
    moe.moe_grouped_gemm_fp8_block(g, *good)
    for i, bad, err in ((0, u8(31, 48), ValueError), (0, torch.zeros((32, 48), device="cuda"), TypeError),
                        (0, u8(48, 32).t(), ValueError), (0, u8(32, 48).cpu(), ValueError),
                        (1, u8(32, 3), ValueError), (1, torch.ones((32, 4), device="cuda"), TypeError),
                        (3, off.long(), TypeError), (3, None, ValueError), (4, u8(1, 32, 48), ValueError),
                        (5, u8(1, 1, 1), ValueError), (6, torch.zeros((32, 32), device="cuda").half(), TypeError),
                        (6, torch.zeros((31, 32), device="cuda"), ValueError)):
        args = list(good)
        args[i] = bad
        with pytest.raises(err):
            moe.moe_grouped_gemm_fp8_block(g, *args)
    x, w = torch.zeros((4, 64), device="cuda"), torch.zeros(64, device="cuda")
    for bad in (lambda: moe.moe_norm(x[0], w, None, 1e-6, x), lambda: moe.moe_norm(x, w.double(), None, 1e-6, x),
                lambda: moe.moe_norm(x, w[:32], None, 1e-6, x), lambda: moe.moe_norm(x.t(), w, None, 1e-6, x),
                lambda: moe.moe_norm(x, w, None, 1e-6, x[:3]), lambda: moe.moe_norm(x, w, None, 1e-6, x, w[:7])):
        with pytest.raises((ValueError, TypeError)):
            bad()
    with pytest.raises(moe.MoEError):
        moe.moe_norm(x, w, None, 0.0, x)
    torch.cuda.synchronize()
    # a stream of its own: the call runs there
    s = torch.cuda.Stream()
    out = torch.full((4, 64), NAN, device="cuda")
    s.wait_stream(torch.cuda.current_stream())
    moe.moe_norm(x + 1, torch.ones(64, device="cuda"), None, 1e-6, out, stream=s)
    s.synchronize()
    assert float((out - 1).abs().max()) < 1e-5
