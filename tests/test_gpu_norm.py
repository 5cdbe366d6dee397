"""The norm and its gradient on the GPU against 64 bits, against differences,
over lengths, types, centred and not; replayed from a graph.

Tolerances.  A sum of n fp32 terms, added in any order, is off by at most n
2^-24 of the sum of magnitudes; the kernels add at most 24 + 6 + 4 + ... terms one
after the other (64 values in a lane, 6 steps over a wave, 4 waves), so 80
2^-24 is taken for a row and (rows in a group + 512) 2^-24 for a column."""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
NAN = float("nan")
U = 2.0 ** -24


@pytest.fixture(scope="module")
def moe():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    from group_limited_routing_router_amd import moe as m
    m.load_library()
    return m


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


SIZES = [(1, 8), (1, 64), (3, 72), (5, 512), (4, 520), (130, 1000), (2, 2048), (7, 2056), (33, 5120), (3, 6144),
         (2, 6152), (5, 16384), (1501, 1000), (600, 64), (2100, 256)]


def inputs(rows, H, x_dtype, dy_dtype, seed, center):
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn((rows, H), generator=gen) * torch.exp(0.7 * torch.randn((rows, 1), generator=gen))
    if center:
        x += 3 * torch.randn((rows, 1), generator=gen)
    w = 1 + 0.1 * torch.randn((H,), generator=gen)
    b = 0.1 * torch.randn((H,), generator=gen)
    dy = torch.randn((rows, H), generator=gen) * 1e-2
    return x.to(x_dtype).cuda(), w.cuda(), b.cuda(), dy.to(dy_dtype).cuda()


def forward64(x, w, b, eps, center):
    mean = x.mean(dim=1, keepdim=True) if center else torch.zeros_like(x[:, :1])
    r = ((x - mean).square().mean(dim=1, keepdim=True) + eps).rsqrt()
    y = (x - mean) * r * w
    return (y if b is None else y + b), mean, r


@pytest.mark.parametrize("center", [False, True], ids=["rms", "layer"])
@pytest.mark.parametrize("x_dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("rows,H", SIZES)
def test_forward(moe, rows, H, x_dtype, center):
    print(f"[case] norm {rows} {H} {x_dtype} {center}", flush=True)
    x, w, b, _ = inputs(rows, H, x_dtype, F32, rows + H, center)
    for out_dtype in (F32, BF16):
        for bias in (None, b):
            out = torch.full((rows + 1, H), NAN, dtype=out_dtype, device="cuda")
            stats = torch.full((rows + 1, 2), NAN, device="cuda")
            moe.moe_norm(x, w, bias, 1e-6, out[:rows], stats[:rows], center=center)
            ref, mean, r = forward64(x.double(), w.double(), None if bias is None else bias.double(), 1e-6, center)
            size = x.double().abs().mean(dim=1, keepdim=True)
            dmean = (80 + 4) * U * size if center else torch.zeros_like(size)
            # r: half of the sum's relative error, the mean's error over the
            # spread, and the steps of the division, root and quotient
            dr = r * (0.5 * 84 * U + r * dmean + 6 * U)
            scaled = (x.double() - mean).abs() * w.double().abs()
            tol = scaled * dr + dmean * r * w.double().abs() + 6 * U * (ref.abs() + scaled * r + b.double().abs())
            tol = tol + half_step(out_dtype) * (ref.abs() + tol) + 1e-30
            assert float(((out[:rows].double() - ref).abs() / tol).max()) <= 1.0
            assert float(((stats[:rows, :1].double() - mean).abs() / (dmean + 1e-30)).max()) <= 1.0
            assert float(((stats[:rows, 1:].double() - r).abs() / dr).max()) <= 1.0
            assert torch.isnan(out[rows]).all() and torch.isnan(stats[rows]).all()


def backward64(dy, x, w, mean, r, center):
    xh = (x - mean) * r
    d = dy * w
    dx = d - xh * (d * xh).mean(dim=1, keepdim=True)
    if center:
        dx = dx - d.mean(dim=1, keepdim=True)
    return dx * r, (dy * xh).sum(dim=0), dy.sum(dim=0)


@pytest.mark.parametrize("center", [False, True], ids=["rms", "layer"])
@pytest.mark.parametrize("types", [(F32, F32), (F32, BF16), (BF16, F32), (BF16, BF16)],
                         ids=lambda t: "-".join("f32" if x == F32 else "bf16" for x in t))
@pytest.mark.parametrize("rows,H", SIZES)
def test_backward(moe, rows, H, types, center):
    print(f"[case] norm backward {rows} {H} {types} {center}", flush=True)
    x, w, b, dy = inputs(rows, H, *types, rows * 3 + H, center)
    _, mean, r = forward64(x.double(), w.double(), None, 1e-6, center)
    stats = torch.cat([mean, r], dim=1).float().contiguous()
    mean, r = stats[:, :1].double(), stats[:, 1:].double()
    ref, rw, rb = backward64(dy.double(), x.double(), w.double(), mean, r, center)
    xh, d = ((x.double() - mean) * r).abs(), (dy.double() * w.double()).abs()
    # xh is off by 3 half steps of its terms, x and mean
    dxh = 3 * U * (x.double().abs() + mean.abs()) * r
    along = (d * xh).mean(dim=1, keepdim=True)
    tol = r * (d * 3 * U + xh * ((90 * U) * along + (d * dxh).mean(dim=1, keepdim=True)) + dxh * along
               + 90 * U * d.mean(dim=1, keepdim=True) + 6 * U * (d + xh * along + d.mean(dim=1, keepdim=True)))
    tw = (rows + 516) * U * (dy.double().abs() * xh).sum(dim=0) + (dy.double().abs() * dxh).sum(dim=0)
    tb = (rows + 512) * U * dy.double().abs().sum(dim=0)
    ws = torch.full((max(16, moe.moe_norm_workspace_bytes(rows, H)),), 0xFF, dtype=torch.uint8, device="cuda")
    for out_dtype in (F32, BF16):
        dx = torch.full((rows + 1, H), NAN, dtype=out_dtype, device="cuda")
        dw, db = torch.full((H + 8,), NAN, device="cuda"), torch.full((H + 8,), NAN, device="cuda")
        moe.moe_norm_backward(dy, x, w, stats, dx[:rows], dw, db, ws, center=center)
        t = tol + half_step(out_dtype) * (ref.abs() + tol) + 1e-30
        assert float(((dx[:rows].double() - ref).abs() / t).max()) <= 1.0
        assert float(((dw[:H].double() - rw).abs() / (tw + 1e-30)).max()) <= 1.0
        assert float(((db[:H].double() - rb).abs() / (tb + 1e-30)).max()) <= 1.0
        assert torch.isnan(dx[rows]).all() and torch.isnan(dw[H:]).all() and torch.isnan(db[H:]).all()
    # added to, without dbias, the same result again
    first = dw[:H].clone()
    more = torch.full((H,), 0.25, device="cuda")
    moe.moe_norm_backward(dy, x, w, stats, dx[:rows], more, None, ws, center=center, accumulate=True)
    assert torch.equal(more, 0.25 + first)


@pytest.mark.parametrize("center", [False, True], ids=["rms", "layer"])
def test_gradient_formula_against_autograd(moe, center):
    gen = torch.Generator().manual_seed(4)
    x, w, b, dy = (torch.randn(s, generator=gen, dtype=torch.float64, requires_grad=True)
                   for s in ((9, 40), (40,), (40,), (9, 40)))
    y, mean, r = forward64(x, w, b, 1e-6, center)
    gx, gw, gb = torch.autograd.grad((y * dy.detach()).sum(), [x, w, b])
    dx, dw, db = backward64(dy.detach(), x.detach(), w.detach(), mean.detach(), r.detach(), center)
    for got, want in ((dx, gx), (dw, gw), (db, gb)):
        assert float((got - want).abs().max()) < 1e-12


@pytest.mark.parametrize("center", [False, True], ids=["rms", "layer"])
def test_gradient_against_differences(moe, center):
    """The kernels' own forward pass (fp32 out) moved along the gradient's
    signs.  A step of 2^-7 of values of about 1 moves the loss by 2^-6 of the
    slope; its fp32 rounding, 2^-22 of terms that add up to a few times the
    slope's, stays below 1e-3 of that, the third order below 1e-3."""
    x, w, b, dy = inputs(6, 200, F32, F32, 12, center)
    dy = dy * 100
    out, stats = torch.empty_like(x), torch.empty((6, 2), device="cuda")
    moe.moe_norm(x, w, b, 1e-6, out, stats, center=center)
    dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty_like(b)
    ws = torch.empty(moe.moe_norm_workspace_bytes(6, 200), dtype=torch.uint8, device="cuda")
    moe.moe_norm_backward(dy, x, w, stats, dx, dw, db, ws, center=center)

    def loss(x, w, b):
        y = torch.empty_like(x)
        moe.moe_norm(x, w, b, 1e-6, y, center=center)
        return float((y.double() * dy.double()).sum())

    t = 2.0 ** -7
    for i, g in enumerate((dx, dw, db)):
        lo, hi = [x, w, b], [x, w, b]
        size = x.abs().mean(dim=1, keepdim=True) if i == 0 else 1.0
        v = torch.sign(g) * size
        lo[i], hi[i] = lo[i] - t * v, hi[i] + t * v
        slope = (loss(*hi) - loss(*lo)) / (2 * t)
        along = float((g.double() * v).sum())
        assert along > 0 and abs(along - slope) <= 0.01 * along, (i, along, slope)


def test_far_mean(moe):
    """A mean of a thousand spreads: the differences keep their digits."""
    gen = torch.Generator().manual_seed(2)
    x = (1000 + torch.randn((4, 4096), generator=gen)).cuda()
    w = torch.ones(4096, device="cuda")
    out = torch.empty_like(x)
    moe.moe_norm(x, w, None, 1e-6, out, center=True)
    ref, mean, r = forward64(x.double(), w.double(), None, 1e-6, True)
    # the mean: 84 half steps of 1000, alike for the whole row
    assert float((out.double() - ref).abs().max()) <= 84 * U * 1000 * 1.1 * 2


def test_zero_and_bad_rows(moe):
    x = torch.randn((5, 520), device="cuda")
    x[1] = 0
    x[2, 7] = float("nan")
    x[3, 9] = float("inf")
    w = torch.ones(520, device="cuda")
    out = torch.empty_like(x)
    moe.moe_norm(x, w, None, 1e-6, out)
    assert (out[1] == 0).all() and torch.isnan(out[2]).all() and torch.isfinite(out[[0, 4]]).all()
    assert not torch.isfinite(out[3, 9])


def test_in_place(moe):
    x = torch.randn((70, 1000), device="cuda")
    w, ws = torch.rand(1000, device="cuda"), torch.empty(moe.moe_norm_workspace_bytes(70, 1000), dtype=torch.uint8,
                                                         device="cuda")
    want, stats = torch.empty_like(x), torch.empty((70, 2), device="cuda")
    moe.moe_norm(x, w, None, 1e-5, want, stats)
    dy, dw = torch.randn_like(x), torch.empty_like(w)
    dx = torch.empty_like(x)
    moe.moe_norm_backward(dy, x, w, stats, dx, dw, None, ws)
    moe.moe_norm_backward(dy, x, w, stats, dy, dw, None, ws)
    assert torch.equal(dy, dx)
    moe.moe_norm(x, w, None, 1e-5, x)
    assert torch.equal(x, want)


def test_no_rows(moe):
    w = torch.ones(64, device="cuda")
    e = torch.empty((0, 64), device="cuda")
    moe.moe_norm(e, w, None, 1e-6, e)
    dw, db = torch.full((64,), NAN, device="cuda"), torch.full((64,), 3.0, device="cuda")
    stats = torch.empty((0, 2), device="cuda")
    moe.moe_norm_backward(e, e, w, stats, e, dw, None, None)
    assert (dw == 0).all()
    dw.fill_(2.0)
    moe.moe_norm_backward(e, e, w, stats, e, dw, db, None, accumulate=True)
    assert (dw == 2).all() and (db == 3).all()


def test_graph_replays(moe):
    x, w, b, dy = inputs(300, 1000, F32, BF16, 5, True)
    out, stats = torch.empty_like(x), torch.empty((300, 2), device="cuda")
    dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty_like(b)
    ws = torch.empty(moe.moe_norm_workspace_bytes(300, 1000), dtype=torch.uint8, device="cuda")

    def step():
        moe.moe_norm(x, w, b, 1e-6, out, stats, center=True)
        moe.moe_norm_backward(dy, x, w, stats, dx, dw, db, ws, center=True)

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for i in range(4):
        x.copy_(torch.randn_like(x) + i)
        step()
        want = [t.clone() for t in (out, stats, dx, dw, db)]
        for t in (out, stats, dx, dw, db):
            t.fill_(NAN)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for t, u in zip((out, stats, dx, dw, db), want):
            assert torch.equal(t, u)
