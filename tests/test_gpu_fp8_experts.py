"""The experts in FP8 by blocks on the GPU: the gated products against 64 bits,
the pass and the block against the calls they are made of, bit for bit, the
gradients against the formulas, automatic differentiation and slopes; rows of
no expert, dense layers, streams, graphs, one training step."""
import pytest
import torch

import _fp8block as f8
from _grouped import counts_for, offsets_of

import numpy as np

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
NAN = float("nan")
NAMES = ("gate", "up", "down")


@pytest.fixture(scope="module")
def moe():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    from group_limited_routing_router_amd import moe as m
    m.load_library()
    return m


class Experts:
    """Weights and tokens of one shape; `first` and `behind` of the T k sorted
    positions belong to no expert."""

    def __init__(self, T, k, E, H, I, seed=0, kind="random", first=0, behind=0, size=0.05):
        rng = np.random.default_rng(seed)
        gen = torch.Generator().manual_seed(seed)
        self.T, self.k, self.E, self.H, self.I, self.P = T, k, E, H, I, T * k
        self.counts = counts_for(self.P - first - behind, E, kind, rng)
        self.offsets = offsets_of(self.counts, first)
        self.pairs = torch.from_numpy(rng.permutation(self.P).astype(np.int32))
        self.rows = self.pairs.long() // k
        self.x = torch.randn((T, H), generator=gen).to(BF16)
        self.dy = (0.1 * torch.randn((self.P, H), generator=gen)).to(BF16)
        self.q, self.s, self.w = {}, {}, {}
        for name, N, K in (("gate", I, H), ("up", I, H), ("down", H, I)):
            w = (size * torch.randn((E, N, K), generator=gen)).to(BF16)
            self.q[name], self.s[name] = f8.quantise_weights(w)
            self.w[name] = f8.value_weights(self.q[name], self.s[name])

    def problem(self, moe):
        return moe.MoEProblem(self.T, self.H, self.I, self.E, 1, 1, self.k, 1.0)

    def weights(self):
        return [t[n].cuda() for n in NAMES for t in (self.q, self.s)]

    def dispatch(self):
        return self.pairs.cuda(), self.offsets.cuda()

    def spans(self):
        off = self.offsets.tolist()
        return [(e, off[e], off[e + 1]) for e in range(self.E) if off[e + 1] > off[e]]

    def owned(self):
        m = torch.zeros(self.P, dtype=torch.bool)
        m[int(self.offsets[0]):int(self.offsets[-1])] = True
        return m

    def gated(self):
        """g and u [P,I] in 64 bits and how far the kernel's may be off."""
        xq = f8.value_rows(*f8.quantise_rows(self.x))[self.rows]
        out = [torch.zeros((self.P, self.I), dtype=torch.float64) for _ in range(4)]
        for e, i, j in self.spans():
            for n, name in enumerate(("gate", "up")):
                out[2 * n][i:j] = xq[i:j] @ self.w[name][e].T
                out[2 * n + 1][i:j] = xq[i:j].abs() @ self.w[name][e].T.abs()
        g, gm, u, um = out
        return g, f8.tolerance(g, gm, self.H, F32), u, f8.tolerance(u, um, self.H, F32)


def sigmoid(g):
    return 1 / (1 + torch.exp(-g))


def gate_up(moe, c, stream=None):
    """x quantised and the gated kernel: h's codes and scales (0x55 where
    nothing is written)."""
    p = c.problem(moe)
    xq = torch.empty((c.T, c.H), dtype=torch.uint8, device="cuda")
    xs = torch.empty((c.T, f8.pitch(c.H)), dtype=torch.uint8, device="cuda")
    moe.moe_quantize_rows_fp8_block(c.x.cuda(), xq, xs, stream=stream)
    h = torch.full((c.P + 1, c.I), 0x55, dtype=torch.uint8, device="cuda")
    hs = torch.full((c.P + 1, f8.pitch(c.I)), 0x55, dtype=torch.uint8, device="cuda")
    moe.moe_expert_gate_up_fp8_block(p, xq, xs, *c.dispatch(), *c.weights()[:4], h[:c.P], hs[:c.P], stream=stream)
    torch.cuda.synchronize()
    assert (h[c.P] == 0x55).all() and (hs[c.P] == 0x55).all()
    return h[:c.P], hs[:c.P]


SHAPES = [
    # T, k, E, H, I
    (1, 1, 1, 128, 64),
    (3, 2, 4, 256, 64),
    (40, 2, 3, 128, 320),
    (130, 4, 5, 384, 192),
    (300, 1, 2, 640, 704),
    (257, 2, 2, 512, 128),
    (64, 8, 16, 256, 448),
    (9, 1, 1, 5120, 384),
]
IDS = ["x".join(map(str, s)) for s in SHAPES]


def build(shape, seed, **kw):
    T, k, E, H, I = shape
    few = T * k > 20
    return Experts(T, k, E, H, I, seed=seed, first=2 if few else 0, behind=5 if few else 0, **kw)


@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_gate_up(moe, shape):
    """h as codes: within half a step of e4m3 of the 64-bit h (half a step of
    the smallest codes below), beside what g and u are off and 20 half steps of
    fp32 for the activation (expf 2, the division and products 4, the sum 1,
    each counted on a sigmoid whose derivative is at most the value)."""
    print(f"[case] gate_up {shape}", flush=True)
    c = build(shape, 1)
    h, hs = gate_up(moe, c)
    own = c.owned()
    assert (h.cpu()[~own] == 0x55).all() and (hs.cpu()[~own] == 0x55).all()
    got = f8.value_rows(h.cpu()[own], hs.cpu()[own])
    g, tg, u, tu = (t[own] for t in c.gated())
    s = sigmoid(g)
    ref = g * s * u
    # d silu / d g is at most 1.1
    off = 1.1 * tg * u.abs() + (g * s).abs() * tu + 1.1 * tg * tu + 20 * 2.0 ** -24 * ref.abs()
    top = torch.nn.functional.pad(ref.abs() + off, (0, -c.I % 128)).reshape(len(ref), -1, 128).amax(2)
    e, _, _ = f8.scale_exponents(top)
    scale = torch.exp2(e).repeat_interleave(128, 1)[:, :c.I]
    tol = 2.0 ** -4 * (ref.abs() + off) + 2.0 ** -10 * scale + off
    assert float(((got - ref).abs() / tol).max()) <= 1.0
    # the scales: those of the block's largest magnitude, give or take what it is off
    low, _, _ = f8.scale_exponents(torch.nn.functional.pad((ref.abs() - off).clamp(min=0), (0, -c.I % 128))
                                   .reshape(len(ref), -1, 128).amax(2))
    used = hs.cpu()[own][:, :f8.blocks(c.I)].double() - 127
    assert (used <= e).all() and (used >= low).all()


def ffn(moe, c, dtype, stream=None, dispatch=None):
    p = c.problem(moe)
    ws = torch.full((moe.moe_fp8_block_workspace_bytes(p),), 0xFF, dtype=torch.uint8, device="cuda")
    y = torch.full((c.P, c.H), NAN, dtype=dtype, device="cuda")
    moe.moe_expert_ffn_fp8_block(p, c.x.cuda(), *(c.dispatch() if dispatch is None else dispatch), *c.weights(), y, ws,
                                 stream=stream)
    torch.cuda.synchronize()
    return y


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_ffn_is_its_calls(moe, shape, dtype):
    """Quantise, gate_up and the product, bit for bit."""
    print(f"[case] ffn {shape}", flush=True)
    c = build(shape, 2)
    y = ffn(moe, c, dtype)
    h, hs = gate_up(moe, c)
    g = moe.MoEGemmProblem(c.P, c.P, c.E, c.H, c.I, 1)
    want = torch.full((c.P, c.H), NAN, dtype=dtype, device="cuda")
    ws = torch.full((max(16, moe.moe_gemm_workspace_bytes(g)),), 0xFF, dtype=torch.uint8, device="cuda")
    moe.moe_grouped_gemm_fp8_block(g, h, hs, None, c.offsets.cuda(), c.q["down"].cuda(), c.s["down"].cuda(), want, ws)
    torch.cuda.synchronize()
    own = c.owned().cuda()
    assert torch.equal(y[own], want[own]) and torch.isnan(y[~own]).all() and torch.isfinite(y[own]).all()


def test_dense_layer_without_dispatch(moe):
    c = Experts(70, 1, 1, 256, 192, seed=3)
    c.pairs = torch.arange(70, dtype=torch.int32)
    c.rows = c.pairs.long()
    assert torch.equal(ffn(moe, c, F32, dispatch=(None, None)), ffn(moe, c, F32))


def test_nan_token(moe):
    """A token with a NaN or an infinity has NaN in its own outputs alone."""
    c = Experts(50, 2, 4, 256, 192, seed=4)
    clean = ffn(moe, c, F32)
    c.x[7, 3], c.x[9, 200] = NAN, float("inf")
    y = ffn(moe, c, F32)
    bad = ((c.rows == 7) | (c.rows == 9)).cuda()
    assert torch.isnan(y[bad]).all() and torch.equal(y[~bad], clean[~bad])


def test_zero_tokens_and_far_gates(moe):
    """Rows of zeros give zeros; gates of -200 and 200 neither overflow nor lose
    the sign."""
    c = Experts(40, 1, 2, 128, 128, seed=5, size=3.0)
    c.x[3] = 0
    c.x[4:20] *= 4
    y = ffn(moe, c, F32)
    assert (y[c.rows.cuda() == 3] == 0).all() and torch.isfinite(y).all()


# ---- the block ----


@pytest.mark.parametrize("T", [1, 64, 700])
def test_block_is_its_calls(moe, T):
    """Route, permute, the experts, combine: bit for bit."""
    gen = torch.Generator().manual_seed(T)
    c = Experts(T, 4, 16, 256, 192, seed=T)
    p = moe.MoEProblem(T, 256, 192, 16, 4, 2, 4, 2.5)
    x, wr = c.x.cuda(), (0.1 * torch.randn((16, 256), generator=gen)).to(BF16).cuda()
    bias = torch.zeros(16, device="cuda")
    ws = torch.full((moe.moe_fp8_block_workspace_bytes(p),), 0xFF, dtype=torch.uint8, device="cuda")
    y = torch.full((T * 4, 256), NAN, device="cuda")
    got = torch.full((T, 256), NAN, device="cuda")
    ids, wts = torch.empty((T, 4), dtype=torch.int32, device="cuda"), torch.empty((T, 4), device="cuda")
    moe.moe_forward_fp8_block(p, x, wr, bias, *c.weights(), got, ids, wts, y, ws)
    b = moe.alloc_buffers(p)
    moe.moe_route(p, x, wr, bias, b["topk_ids"], b["topk_weights"])
    moe.moe_permute(p, b["topk_ids"], b["expert_offsets"], b["sorted_pairs"], b["pair_rows"], b["ws"])
    moe.moe_expert_ffn_fp8_block(p, x, b["sorted_pairs"], b["expert_offsets"], *c.weights(), b["y"], ws)
    moe.moe_combine(p, b["y"], b["pair_rows"], b["topk_weights"], b["out"])
    torch.cuda.synchronize()
    assert torch.equal(ids, b["topk_ids"]) and torch.equal(wts, b["topk_weights"])
    assert torch.equal(got, b["out"]) and torch.isfinite(got).all()
    half = torch.empty((T, 256), dtype=BF16, device="cuda")
    moe.moe_forward_fp8_block(p, x, wr, None, *c.weights(), half, None, None, y, ws)
    assert torch.equal(half, got.to(BF16))


# ---- gradients ----


def backward(moe, c, dx_dtype=F32, dw_dtype=F32, start=None, ws=None, out=None):
    p = c.problem(moe)
    if ws is None:
        ws = torch.full((moe.moe_fp8_block_backward_workspace_bytes(p),), 0xFF, dtype=torch.uint8, device="cuda")
    if out is None:
        dx = torch.full((c.P, c.H), NAN, dtype=dx_dtype, device="cuda")
        dw = [torch.full(c.q[n].shape, NAN, dtype=dw_dtype, device="cuda") if start is None else start[n].clone()
              for n in NAMES]
    else:
        dx, dw = out
    moe.moe_expert_ffn_fp8_block_backward(p, c.x.cuda(), *c.dispatch(), *c.weights(), c.dy.cuda(), dx, *dw, ws,
                                          accumulate=start is not None)
    return dx, dict(zip(NAMES, dw))


def reference_gradients(c):
    """dx and dw in 64 bits without the kernels' roundings of dy, dg, du and h,
    and a tolerance for each from these roundings."""
    g, tg, u, tu = c.gated()
    s = sigmoid(g)
    silu, slope = g * s, s * (1 + g * (1 - s))
    dyq = f8.value_rows(*f8.quantise_rows(c.dy))
    x = c.x.double()[c.rows]
    dy = c.dy.double()
    zeros = {n: torch.zeros(c.w[n].shape, dtype=torch.float64) for n in NAMES}
    dw, tw = zeros, {n: torch.zeros_like(t) for n, t in zeros.items()}
    dx, tx = torch.zeros((c.P, c.H), dtype=torch.float64), torch.zeros((c.P, c.H), dtype=torch.float64)
    half = 2.0 ** -8  # of bf16

    def rounded(v, off):
        """How far v, off by `off`, is off after its rounding by blocks."""
        top = torch.nn.functional.pad(v.abs() + off, (0, -c.I % 128)).reshape(len(v), -1, 128).amax(2)
        e, _, _ = f8.scale_exponents(top)
        return off + 2.0 ** -4 * (v.abs() + off) + 2.0 ** -10 * torch.exp2(e).repeat_interleave(128, 1)[:, :c.I]

    for e, i, j in c.spans():
        wg, wu, wd = (c.w[n][e] for n in NAMES)
        dh = dyq[i:j] @ wd
        th = f8.tolerance(dh, dyq[i:j].abs() @ wd.abs(), c.H, F32)
        G, U, S, T1, T2 = g[i:j], u[i:j], silu[i:j], tg[i:j], tu[i:j]
        dg, du, h = dh * U * slope[i:j], dh * S, S * U
        # the slope of silu is at most 1.1, its own slope at most 0.5
        og = (th * U.abs() + dh.abs() * T2 + th * T2) * 1.1 + dh.abs() * U.abs() * 0.5 * T1 + 24 * 2.0 ** -24 * dg.abs()
        ou = th * S.abs() + dh.abs() * 1.1 * T1 + th * 1.1 * T1 + 24 * 2.0 ** -24 * du.abs()
        oh = 1.1 * T1 * U.abs() + S.abs() * T2 + 1.1 * T1 * T2 + 24 * 2.0 ** -24 * h.abs()
        dx[i:j] = dg @ wg + du @ wu
        mag = dg.abs() @ wg.abs() + du.abs() @ wu.abs()
        rg, ru = rounded(dg, og), rounded(du, ou)
        tx[i:j] = rg @ wg.abs() + ru @ wu.abs()
        tx[i:j] += (f8.CUT + (c.I / 4 + 32) * 2.0 ** -23) * (mag + tx[i:j])
        rows = j - i
        sums = (rows / 16 + 32) * 2.0 ** -23
        for n, left, off, right, roff in (("gate", dg, og, x[i:j], 0), ("up", du, ou, x[i:j], 0),
                                          ("down", dy[i:j], 0, h, oh)):
            lo = off + half * (left.abs() + off) if n != "down" else torch.zeros_like(left)
            ro = roff + half * (right.abs() + roff) if n == "down" else torch.zeros_like(right)
            dw[n][e] = left.T @ right
            t = lo.T @ right.abs() + left.abs().T @ ro + lo.T @ ro
            tw[n][e] = t + sums * (left.abs().T @ right.abs() + t)
    return dx, tx, dw, tw


def within(got, ref, tol, dtype):
    t = tol + torch.finfo(dtype).eps / 2 * (ref.abs() + tol) + 1e-30
    x = ((got.cpu().double() - ref).abs() / t)
    return float(torch.nan_to_num(x, nan=float("inf")).max()) if x.numel() else 0.0


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_gradients(moe, shape, dtype):
    print(f"[case] gradients {shape} {dtype}", flush=True)
    c = build(shape, 6)
    dx, dw = backward(moe, c, dtype, dtype)
    torch.cuda.synchronize()
    rdx, tx, rdw, tw = reference_gradients(c)
    own = c.owned()
    assert torch.isnan(dx.cpu()[~own]).all()
    assert within(dx[own.cuda()], rdx[own], tx[own], dtype) <= 1.0
    for n in NAMES:
        assert within(dw[n], rdw[n], tw[n], dtype) <= 1.0, n


def test_gradients_add(moe):
    c = build(SHAPES[3], 7)
    _, plain = backward(moe, c)
    start = {n: torch.randn(c.q[n].shape, device="cuda") for n in NAMES}
    _, added = backward(moe, c, start=start)
    torch.cuda.synchronize()
    for n in NAMES:
        want = start[n].double() + plain[n].double()
        # the parts of a split sum are added one by one
        assert float((added[n].double() - want).abs().max()) <= 2.0 ** -22 * float(
            (start[n].abs() + plain[n].abs()).max())


def test_reference_against_autograd():
    """The formulas, without the roundings, in 64 bits on the CPU."""
    c = Experts(12, 2, 3, 128, 64, seed=8)
    x = c.x.double()[c.rows].requires_grad_()
    w = {n: c.w[n].clone().requires_grad_() for n in NAMES}
    total = 0.0
    dyq = f8.value_rows(*f8.quantise_rows(c.dy))
    for e, i, j in c.spans():
        g, u = x[i:j] @ w["gate"][e].T, x[i:j] @ w["up"][e].T
        total = total + (dyq[i:j] * ((g * sigmoid(g) * u) @ w["down"][e].T)).sum()
    grads = torch.autograd.grad(total, [x, *w.values()])
    # the reference with x and dy as they are quantised
    c.dy = dyq
    quantised = c.gated
    xs = c.x.double()[c.rows]

    def unrounded():
        _, tg, _, tu = quantised()
        g, u = torch.zeros_like(tg), torch.zeros_like(tu)
        for e, i, j in c.spans():
            g[i:j], u[i:j] = xs[i:j] @ c.w["gate"][e].T, xs[i:j] @ c.w["up"][e].T
        return g, tg, u, tu
    c.gated = unrounded
    rdx, _, rdw, _ = reference_gradients(c)
    for got, want in zip((rdx, *rdw.values()), grads):
        assert float((got - want).abs().max()) <= 2.0 ** -40 * float(want.abs().max())


@pytest.mark.parametrize("shape", SHAPES[1:6], ids=IDS[1:6])
def test_gradients_along_their_signs(moe, shape):
    """The kernels' gradients along the signs of the 64-bit slope of the
    unrounded pass.  Rounding operands to e4m3 moves each term by up to 2^-4,
    either way: a sum of many gradients stays within a tenth, and zeros, halves
    and other signs do not."""
    c = build(shape, 9)
    dx, dw = backward(moe, c)
    torch.cuda.synchronize()
    x = torch.where(c.owned()[:, None], c.x.double()[c.rows], 0).requires_grad_()
    w = {n: c.w[n].clone().requires_grad_() for n in NAMES}
    total = 0.0
    for e, i, j in c.spans():
        g, u = x[i:j] @ w["gate"][e].T, x[i:j] @ w["up"][e].T
        total = total + (c.dy.double()[i:j] * ((g * sigmoid(g) * u) @ w["down"][e].T)).sum()
    grads = torch.autograd.grad(total, [x, *w.values()])
    for got, want in zip((dx, *dw.values()), grads):
        slope = float(want.abs().sum())
        along = float((got.cpu().double().nan_to_num(nan=0.0) * torch.sign(want)).sum())
        assert abs(along - slope) <= 0.1 * slope


def test_no_tokens(moe):
    c = Experts(0, 1, 2, 128, 64, seed=1)
    p = c.problem(moe)
    c.offsets = torch.zeros(3, dtype=torch.int32)
    dw = [torch.full(c.q[n].shape, NAN, device="cuda") for n in NAMES]
    ws = torch.empty((max(16, moe.moe_fp8_block_backward_workspace_bytes(p)),), dtype=torch.uint8, device="cuda")
    moe.moe_expert_ffn_fp8_block_backward(p, None, None, c.offsets.cuda(), *c.weights(), None, None, *dw, ws)
    assert all((t == 0).all() for t in dw)


# ---- use ----


def test_graph_replays(moe):
    """Forward and backward captured together and replayed with other tokens."""
    c = build(SHAPES[3], 10)
    p = c.problem(moe)
    x, dy, disp, w = c.x.cuda(), c.dy.cuda(), c.dispatch(), c.weights()
    ws = torch.empty(moe.moe_fp8_block_workspace_bytes(p), dtype=torch.uint8, device="cuda")
    wb = torch.empty(moe.moe_fp8_block_backward_workspace_bytes(p), dtype=torch.uint8, device="cuda")
    y, dx = torch.zeros((c.P, c.H), device="cuda"), torch.zeros((c.P, c.H), device="cuda")
    dw = [torch.zeros(c.q[n].shape, dtype=BF16, device="cuda") for n in NAMES]

    def step():
        moe.moe_expert_ffn_fp8_block(p, x, *disp, *w, y, ws)
        moe.moe_expert_ffn_fp8_block_backward(p, x, *disp, *w, dy, dx, *dw, wb)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(4):
        x.copy_(torch.randn(x.shape, device="cuda") * (i + 1))
        step()
        want = [t.clone() for t in (y, dx, *dw)]
        for t in (y, dx, *dw):
            t.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(t, u) for t, u in zip((y, dx, *dw), want))


def test_two_streams(moe):
    a, b = build(SHAPES[3], 11), build(SHAPES[6], 12)
    want = [ffn(moe, c, F32).nan_to_num() for c in (a, b)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    calls = []
    for c in (a, b):
        p = c.problem(moe)
        calls.append((p, c.x.cuda(), *c.dispatch(), *c.weights(), torch.zeros((c.P, c.H), device="cuda"),
                      torch.empty(moe.moe_fp8_block_workspace_bytes(p), dtype=torch.uint8, device="cuda")))
    torch.cuda.synchronize()
    for _ in range(4):
        for args, s in zip(calls, streams):
            moe.moe_expert_ffn_fp8_block(*args, stream=s)
    torch.cuda.synchronize()
    for args, w in zip(calls, want):
        assert torch.equal(args[-2], w)


def test_training_step(moe):
    """The norm, the router, the experts and the combine, and back: every call
    on what the others wrote, against one 64-bit pass with automatic
    differentiation.  The operands' roundings to e4m3 leave the result within a
    tenth in norm, and the gradients on the same side."""
    T, k, E, H, I = 96, 2, 8, 256, 192
    gen = torch.Generator().manual_seed(13)
    c = Experts(T, k, E, H, I, seed=13)
    p = moe.MoEProblem(T, H, I, E, 4, 2, k, 2.5)
    stream_x = (2 * torch.randn((T, H), generator=gen)).cuda()
    weight = (1 + 0.1 * torch.randn((H,), generator=gen)).cuda()
    wr = (0.1 * torch.randn((E, H), generator=gen)).to(BF16).cuda()
    x, stats = torch.empty((T, H), dtype=BF16, device="cuda"), torch.empty((T, 2), device="cuda")
    moe.moe_norm(stream_x, weight, None, 1e-6, x, stats)
    b = moe.alloc_buffers(p)
    ws = torch.empty(moe.moe_fp8_block_workspace_bytes(p), dtype=torch.uint8, device="cuda")
    moe.moe_forward_fp8_block(p, x, wr, None, *c.weights(), b["out"], b["topk_ids"], b["topk_weights"], b["y"], ws)
    moe.moe_permute(p, b["topk_ids"], b["expert_offsets"], b["sorted_pairs"], b["pair_rows"], b["ws"])
    dout = torch.randn((T, H), generator=gen).cuda()
    pairs = b["sorted_pairs"].long()
    wts = b["topk_weights"].flatten()[pairs]
    dy = (2.5 * wts[:, None] * dout[pairs // k]).to(BF16)
    dxp = torch.empty((T * k, H), device="cuda")
    dw = [torch.empty(c.q[n].shape, device="cuda") for n in NAMES]
    wb = torch.empty(moe.moe_fp8_block_backward_workspace_bytes(p), dtype=torch.uint8, device="cuda")
    moe.moe_expert_ffn_fp8_block_backward(p, x, b["sorted_pairs"], b["expert_offsets"], *c.weights(), dy, dxp, *dw, wb)
    ones = moe.MoEProblem(T, H, I, E, 4, 2, k, 1.0)
    dx = torch.empty((T, H), device="cuda")
    moe.moe_combine(ones, dxp, b["pair_rows"], torch.ones((T, k), device="cuda"), dx)
    dstream, dweight = torch.empty_like(stream_x), torch.empty_like(weight)
    wn = torch.empty(moe.moe_norm_workspace_bytes(T, H), dtype=torch.uint8, device="cuda")
    moe.moe_norm_backward(dx, stream_x, weight, stats, dstream, dweight, None, wn)
    torch.cuda.synchronize()

    leaves = [stream_x.double().cpu().requires_grad_(), weight.double().cpu().requires_grad_(),
              *(c.w[n].clone().requires_grad_() for n in NAMES)]
    s, wt, wg, wu, wd = leaves
    xn = s * (s.square().mean(1, keepdim=True) + 1e-6).rsqrt() * wt
    out = torch.zeros((T, H), dtype=torch.float64)
    ids, tw = b["topk_ids"].cpu(), b["topk_weights"].double().cpu()
    for e in range(E):
        t, j = (ids == e).nonzero(as_tuple=True)
        g, u = xn[t] @ wg[e].T, xn[t] @ wu[e].T
        out = out.index_add(0, t, 2.5 * tw[t, j][:, None] * ((g * sigmoid(g) * u) @ wd[e].T))
    want = torch.autograd.grad((out * dout.double().cpu()).sum(), leaves)
    for got, ref in zip((b["out"], dstream, dweight, *dw), (out.detach(), *want)):
        assert float((got.double().cpu() - ref).norm() / ref.norm()) < 0.1
