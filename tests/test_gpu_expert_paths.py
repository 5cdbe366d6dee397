"""The int8 block and the experts' gradients as whole calls: at the block's own
sizes (hidden 5120, intermediate 2560, 256 experts, 8 for each token) and
captured into graphs."""
import pytest
import torch

from group_limited_routing_router_amd.inputs import CONFIGS, MoEConfig

from _grouped import worst
from test_gpu_grouped_experts import SHAPES, quantized, reference_gradients, setup

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    from group_limited_routing_router_amd import moe as m
    m.load_library()
    yield m
    torch.cuda.empty_cache()


def block(T):
    c = CONFIGS["decode"]
    return MoEConfig("block", T=T, H=c.H, I=c.I, E=c.E, G=c.G, TG=c.TG, k=c.k, scale=c.scale)


def normal(shape, gen, scale):
    """bf16 normal values drawn on the GPU, an expert at a time."""
    x = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
    for part in (x if len(shape) == 3 else [x]):
        part.copy_(torch.randn(part.shape, generator=gen, device="cuda").mul_(scale))
    return x


def dispatch(moe, cfg, seed):
    """Tokens routed to busy and idle experts: x, the permutation, each
    position's token, each expert's positions."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    p = moe.MoEProblem.from_config(cfg)
    x = normal((cfg.T, cfg.H), gen, 1.0)
    liking = torch.randn((cfg.E,), generator=gen, device="cuda") * 0.7
    ids = (torch.randn((cfg.T, cfg.E), generator=gen, device="cuda") + liking).topk(cfg.k, dim=1).indices
    b = moe.alloc_buffers(p)
    b["topk_ids"].copy_(ids)
    moe.moe_permute(p, b["topk_ids"], b["expert_offsets"], b["sorted_pairs"], b["pair_rows"], b["ws"])
    torch.cuda.synchronize()
    off = b["expert_offsets"].tolist()
    return gen, p, x, b, b["sorted_pairs"].long() // cfg.k, [(off[e], off[e + 1]) for e in range(cfg.E)]


def some_experts(spans):
    """The first, the last, the busiest and the least busy expert with rows, and three more."""
    filled = [e for e, (i, j) in enumerate(spans) if j > i]
    by_rows = sorted(filled, key=lambda e: spans[e][1] - spans[e][0])
    return sorted({filled[0], filled[-1], by_rows[0], by_rows[-1], *filled[len(filled) // 4::len(filled) // 4]})


@pytest.mark.parametrize("T", [128, 8192])
def test_int8_block(moe, T):
    """y of some experts against the definition in 64 bits, with the tolerance
    of h's codes: h is off by at most 2^-20 of itself, so a code within 127
    2^-19 of a half way point may be the next one; 2^-19 of the value for the
    scales and the last roundings.  Then the whole pass, from its own routing,
    against its steps, bit for bit."""
    print(f"[case] int8 block, {T} tokens", flush=True)
    cfg = block(T)
    gen, p, x, b, rows, spans = dispatch(moe, cfg, 3)
    E, H, I = cfg.E, cfg.H, cfg.I

    def weights(shape):
        w = torch.empty(shape, dtype=torch.int8, device="cuda")
        for part in w:
            part.copy_(torch.randn(part.shape, generator=gen, device="cuda").mul_(32).round_().clamp_(-127, 127))
        return w, torch.rand(shape[:2], generator=gen, device="cuda") * 4e-4 + 4e-4
    (qg, sg), (qu, su), (qd, sd) = weights((E, I, H)), weights((E, I, H)), weights((E, H, I))
    ws = torch.full((moe.moe_int8_workspace_bytes(p),), 0xFF, dtype=torch.uint8, device="cuda")
    y = torch.full((T * cfg.k, H), float("nan"), device="cuda")
    moe.moe_expert_ffn_int8(p, x, b["sorted_pairs"], b["expert_offsets"], qg, sg, qu, su, qd, sd, y, ws)
    xc = torch.empty((T, H), dtype=torch.int8, device="cuda")
    xs = torch.empty((T,), device="cuda")
    moe.moe_quantize_rows_int8(x, xc, xs)
    torch.cuda.synchronize()
    assert bool(torch.isfinite(y).all())
    for e in some_experts(spans):
        i, j = spans[e]
        a, s = xc[rows[i:j]].double(), xs[rows[i:j]][:, None]
        g = ((a @ qg[e].double().T).float() * (s * sg[e])).double()
        u = ((a @ qu[e].double().T).float() * (s * su[e])).double()
        h = g / (1 + torch.exp(-g)) * u
        amax = h.abs().amax(dim=1, keepdim=True)
        v = 127 * h / amax
        code = torch.round(v)
        near = ((v - torch.floor(v) - 0.5).abs() < 127 * 2.0 ** -19).double()
        step, d = (amax / 127) * sd[e].double(), qd[e].double()
        tol = near @ d.abs().T * step + 2.0 ** -19 * (code.abs() @ d.abs().T * step)
        w = worst(y[i:j], code @ d.T * step, tol + 1e-30)
        assert w <= 1.0, f"expert {e}, {j - i} rows: {w:.3g} of the tolerance"
    w_router = normal((E, H), gen, 0.02)
    bias = torch.randn((E,), generator=gen, device="cuda") * 0.1
    moe.moe_route(p, x, w_router, bias, b["topk_ids"], b["topk_weights"])
    moe.moe_permute(p, b["topk_ids"], b["expert_offsets"], b["sorted_pairs"], b["pair_rows"], b["ws"])
    moe.moe_expert_ffn_int8(p, x, b["sorted_pairs"], b["expert_offsets"], qg, sg, qu, su, qd, sd, y, ws)
    ref = torch.full((T, H), float("nan"), dtype=torch.bfloat16, device="cuda")
    moe.moe_combine(p, y, b["pair_rows"], b["topk_weights"], ref)
    out, y2 = torch.full_like(ref, float("nan")), torch.full_like(y, float("nan"))
    ws.fill_(0xFF)
    moe.moe_forward_int8(p, x, w_router, bias, qg, sg, qu, su, qd, sd, out, None, None, y2, ws)
    torch.cuda.synchronize()
    assert torch.equal(y2, y) and torch.equal(out, ref)


@pytest.mark.parametrize("T,dtype,accumulate", [(128, torch.float32, False), (128, torch.float32, True),
                                                (8192, torch.bfloat16, False)],
                         ids=["T128_f32", "T128_f32_adding", "T8192_bf16"])
def test_block_gradients(moe, T, dtype, accumulate):
    """Some experts' gradients against 64 bits (tolerances of
    reference_gradients), the idle experts' all zero (or as they were)."""
    print(f"[case] gradients of the block, {T} tokens, {dtype}, accumulate {accumulate}", flush=True)
    cfg = block(T)
    gen, p, x, b, rows, spans = dispatch(moe, cfg, 4)
    E, H, I, P = cfg.E, cfg.H, cfg.I, cfg.T * cfg.k
    w = {"w_gate": normal((E, I, H), gen, 0.02), "w_up": normal((E, I, H), gen, 0.02),
         "w_down": normal((E, H, I), gen, 0.02)}
    dy = normal((P, H), gen, 1.0)
    dx = torch.full((P, H), float("nan"), device="cuda")
    start = 3.0 if accumulate else float("nan")
    dw = {n: torch.full(t.shape, start, dtype=dtype, device="cuda") for n, t in w.items()}
    ws = torch.full((moe.moe_backward_workspace_bytes(p),), 0xFF, dtype=torch.uint8, device="cuda")
    moe.moe_expert_ffn_backward(p, x, b["sorted_pairs"], b["expert_offsets"], w["w_gate"], w["w_up"], w["w_down"],
                                dy, dx, dw["w_gate"], dw["w_up"], dw["w_down"], ws, accumulate=accumulate)
    torch.cuda.synchronize()
    assert bool(torch.isfinite(dx).all())
    last = 2.0 ** -8 * 1.01 if dtype == torch.bfloat16 else 0.0
    base = 3.0 if accumulate else 0.0
    for e in some_experts(spans):
        i, j = spans[e]
        one = MoEConfig("one", T=j - i, H=H, I=I, E=1, G=1, TG=1, k=1, scale=1.0)
        d = {"x": x[rows[i:j]], **{n: t[e:e + 1] for n, t in w.items()}}
        rdx, rdw = reference_gradients(one, d, torch.arange(j - i, device="cuda"), [(0, 0, j - i)], dy[i:j])
        assert worst(dx[i:j], rdx[0], rdx[1] + 1e-30) <= 1.0, e
        for n, (v, t) in rdw.items():
            v, t = v[0] + base, t[0] + 2.0 ** -24 * (base + (v[0] + base).abs())
            r = worst(dw[n][e], v, t + last * v.abs() + 1e-30)
            assert r <= 1.0, f"d{n} of expert {e}, {j - i} rows: {r:.3g} of the tolerance"
        del rdx, rdw
    for e, (i, j) in enumerate(spans):
        if i == j:
            assert all(bool((t[e] == base).all()) for t in dw.values()), e


@pytest.mark.parametrize("shape", [SHAPES[2], SHAPES[4]], ids=lambda s: "T%d_H%d_I%d_E%d_k%d" % (*s[:4], s[6]))
def test_paths_replayed(moe, shape):
    """The int8 pass and the gradients captured together, replayed with other
    tokens in the same buffers and eager work between; every replay against the
    eager calls."""
    print(f"[case] replays {shape}", flush=True)
    cases = [setup(moe, shape, s) for s in (71, 72, 73)]
    cfg, p, d, b, _, _ = cases[0]
    P = cfg.T * cfg.k
    q8 = [t for n in ("w_gate", "w_up", "w_down") for t in quantized(moe, d[n])]
    buf = {"x": d["x"].clone(), "off": b["expert_offsets"].clone(), "pairs": b["sorted_pairs"].clone(),
           "dy": torch.zeros((P, cfg.H), dtype=torch.bfloat16, device="cuda")}
    ws8 = torch.empty((moe.moe_int8_workspace_bytes(p),), dtype=torch.uint8, device="cuda")
    wsb = torch.empty((moe.moe_backward_workspace_bytes(p),), dtype=torch.uint8, device="cuda")

    def outputs():
        def f(*s):
            return torch.full(s, float("nan"), device="cuda")
        return dict(out=f(cfg.T, cfg.H), y=f(P, cfg.H), dx=f(P, cfg.H),
                    **{n: f(*d[n].shape) for n in ("w_gate", "w_up", "w_down")})

    def calls(o):
        moe.moe_forward_int8(p, buf["x"], d["w_router"], d["bias"], *q8, o["out"], None, None, o["y"], ws8)
        moe.moe_expert_ffn_backward(p, buf["x"], buf["pairs"], buf["off"], d["w_gate"], d["w_up"], d["w_down"],
                                    buf["dy"], o["dx"], o["w_gate"], o["w_up"], o["w_down"], wsb)
    o = outputs()
    calls(o)
    torch.cuda.synchronize()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            calls(o)
    torch.cuda.current_stream().wait_stream(side)
    gen = torch.Generator(device="cuda").manual_seed(5)
    for n in range(5):
        _, _, dn, bn, _, _ = cases[n % 3]
        buf["x"].copy_(dn["x"])
        buf["off"].copy_(bn["expert_offsets"])
        buf["pairs"].copy_(bn["sorted_pairs"])
        buf["dy"].copy_(torch.randn((P, cfg.H), generator=gen, device="cuda"))
        ref = outputs()
        calls(ref)
        torch.cuda.synchronize()
        for t in o.values():
            t.fill_(float("nan"))
        ws8.fill_(0xFF)
        wsb.fill_(0xFF)
        graph.replay()
        torch.cuda.synchronize()
        for name in o:
            assert bool(torch.isfinite(ref[name]).all()) and torch.equal(o[name], ref[name]), (n, name)
