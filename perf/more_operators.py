"""Cases of the experts in 8-bit floating point with a scale for each block of
128: their matrix products, their gated feed-forward pass and its gradients,
and the norm that makes the block's input.

FP8 operands are e4m3 codes with scales that are powers of two,

    scale = 2^ceil(log2(amax / 448)),  codes = value / scale to the nearest
                                       e4m3 (ties to even)

(blocks of zeros: scale 1).  A block is 128 values along a row of activations
or gradients (quantised within the pass), or 128 x 128 of a weight matrix
(quantised beforehand; a scale is held as its exponent + 127).  Positions q are
sorted by expert as in operators.py: expert e owns offsets[e] ..
offsets[e + 1], position q belongs to token sorted_pairs[q] // k.

    product     out[q] = A[row(q)] . W[e]^T           A, W: the dequantised operands
    input_grad  da[q]  = D[q] . W[e]
    ffn         g = A . Wgate[e]^T, u = A . Wup[e]^T, h = silu(g) u quantised by
                rows, y[q] = h . Wdown[e]^T
    ffn_grad    from dy: dh = quantised dy . Wdown, dg = dh u s (1 + g (1 - s)),
                du = dh g s with s = 1 / (1 + exp(-g)); dx = (dg quantised) .
                Wgate + (du quantised) . Wup; the weights' gradients dg^T x,
                du^T x and dy^T h by expert from bf16 operands
    norm        out = (x - mean) / sqrt(var + eps) weight + bias by rows; the RMS
                form leaves mean out and takes the mean square for var
    norm_grad   from dy: dx and the gradients of weight and bias

Activations, gradients and the outputs of products are bf16 (beside operands of
4 significant bits), the residual stream that the norm reads fp32 or bf16.
"""
import math

import torch

own = False

# the repository's block: hidden 5120, intermediate 2560, 256 experts, 8 for
# each token; its dense layers have an intermediate size of 20480
HIDDEN, INTER, EXPERTS, TOP = 5120, 2560, 256, 8
BLOCK = 128


def listed():
    block = dict(E=EXPERTS, k=TOP, skew=0.0)
    return [
        # a decode batch: 4 rows for each expert, every weight read once
        dict(name="product decode", op="product", T=128, N=INTER, K=HIDDEN, **block),
        # a prefill chunk: 256 rows for each expert
        dict(name="product prefill", op="product", T=8192, N=INTER, K=HIDDEN, **block),
        # the gradient of the down projection's input, busy and idle experts
        dict(name="input_grad skewed", op="input_grad", T=4096, k=TOP, E=EXPERTS, N=HIDDEN, K=INTER, skew=0.7),
        # few experts, sizes that end inside a block, rows in sorted order
        dict(name="input_grad odd", op="input_grad", T=5003, k=1, E=24, N=1008, K=784, skew=0.5),
        # a dense layer for one token: a launch's latency and the weights once
        dict(name="ffn one token", op="ffn", T=1, k=1, E=1, H=HIDDEN, I=20480, skew=0.0),
        # the experts of a prefill chunk
        dict(name="ffn prefill", op="ffn", T=8192, H=HIDDEN, I=INTER, **block),
        # a training step's backward pass at the block's size
        dict(name="ffn_grad chunk", op="ffn_grad", T=4096, H=HIDDEN, I=INTER, **block),
        # few experts of unequal load, sizes that end inside a block
        dict(name="ffn_grad odd", op="ffn_grad", T=901, k=2, E=8, H=1152, I=704, skew=0.5),
        # the smallest call: the pre-norm of a decode batch's residual stream
        dict(name="norm decode", op="norm", rows=128, H=HIDDEN, x="f32", center=False),
        # the pre-norm of a long prefill chunk
        dict(name="norm prefill", op="norm", rows=65536, H=HIDDEN, x="f32", center=False),
        # its gradient in a training step
        dict(name="norm_grad chunk", op="norm_grad", rows=8192, H=HIDDEN, x="f32", center=False),
        # a layer norm with its mean and bias over rows of another size
        dict(name="norm_grad layer odd", op="norm_grad", rows=1501, H=1000, x="bf16", center=True),
    ]


def _between(rng, low, high, step=1):
    """A whole number of [low, high], even over its logarithm, a multiple of step."""
    return max(low, int(math.exp(rng.uniform(math.log(low), math.log(high + 1)))) // step * step)


def draw(rng):
    op = rng.choice(["product", "input_grad", "ffn", "ffn_grad", "norm", "norm_grad"])
    if op in ("norm", "norm_grad"):
        H = _between(rng, 64, 16384, 8)
        rows = _between(rng, 1, min(65536, (65536 if op == "norm" else 16384) * HIDDEN // H))
        return dict(op=op, rows=rows, H=H, x=rng.choice(["f32", "bf16"]), center=rng.choice([False, True]))
    E = _between(rng, 1, EXPERTS)
    k = 1 if op == "input_grad" else min(E, rng.choice([1, 1, 2, 4, 8]))
    T = _between(rng, 1, 65536 // k)
    skew = rng.choice([0.0, 0.3, 0.7, 1.0])
    if op in ("ffn", "ffn_grad"):
        H, I = _between(rng, 128, 8192, 128), _between(rng, 64, 20480, 64)
        while E * H * I > EXPERTS * INTER * HIDDEN:
            H, I = max(128, H // 2 // 128 * 128), max(64, I // 2 // 64 * 64)
        while T * k * H * I > (8192 if op == "ffn" else 4096) * TOP * INTER * HIDDEN:
            T = max(1, T // 2)
        return dict(op=op, T=T, k=k, E=E, H=H, I=I, skew=skew)
    N, K = (_between(rng, 64, 20480, 16) for _ in range(2))
    while E * N * K > EXPERTS * INTER * HIDDEN:
        N, K = max(64, N // 2 // 16 * 16), max(64, K // 2 // 16 * 16)
    while T * k * N * K > 8192 * TOP * INTER * HIDDEN:
        T = max(1, T // 2)
    return dict(op=op, T=T, k=k, E=E, N=N, K=K, skew=skew)


# ---- quantisation, for the inputs and the plain form ----


def _exponents(amax):
    """e with 2^e = the scale of blocks whose largest magnitude is amax."""
    m, e = torch.frexp(amax)  # amax = m 2^e, 448 = 0.875 2^9
    return torch.where(amax > 0, e - 9 + (m > 0.875).to(e.dtype), torch.zeros_like(e))


def _power(e):
    """2^e, exactly, for -127 < e < 128."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _fp8(x):
    """fp32 values of at most 448 rounded to e4m3."""
    return x.to(torch.float8_e4m3fn)


def _padded(x):
    """x [R, C] with C filled up to whole blocks, as [R, blocks, 128]."""
    x = torch.nn.functional.pad(x, (0, -x.shape[1] % BLOCK))
    return x.reshape(x.shape[0], x.shape[1] // BLOCK, BLOCK)


def _rounded_rows(x):
    """The rows of x quantised by blocks and dequantised, in fp32."""
    p = _padded(x)
    e = _exponents(p.abs().amax(dim=2, keepdim=True))
    return (_fp8(p * _power(-e)).float() * _power(e)).reshape(p.shape[0], p.shape[1] * BLOCK)[:, : x.shape[1]]


def _spread(s, rows, cols):
    """A scale for each value from the scales of 128 x 128 blocks."""
    return s.repeat_interleave(BLOCK, 0)[:rows].repeat_interleave(BLOCK, 1)[:, :cols]


def _weights(s, name, e):
    """Weight matrix e of a stack, dequantised, in fp32."""
    w, scales = s["q_" + name][e], s["s_" + name][e]
    return w.float() * _spread(_power(scales.int() - 127), *w.shape)


# ---- inputs ----


def _stack(E, N, K, gen):
    """A stack of FP8 weight matrices and its scales, a matrix at a time."""
    codes = torch.empty((E, N, K), dtype=torch.float8_e4m3fn, device="cuda")
    scales = torch.empty((E, -(-N // BLOCK), -(-K // BLOCK)), dtype=torch.uint8, device="cuda")
    for i in range(E):
        w = torch.randn((N, K), generator=gen, device="cuda").mul_(0.02).bfloat16().float()
        p = torch.nn.functional.pad(w, (0, -K % BLOCK, 0, -N % BLOCK))
        p = p.reshape(scales.shape[1], BLOCK, scales.shape[2], BLOCK)
        e = _exponents(p.abs().amax(dim=(1, 3)))
        codes[i] = _fp8(w * _spread(_power(-e), N, K))
        scales[i] = (e + 127).to(torch.uint8)
    return codes, scales


def _acts(shape, gen):
    """Activations: a few channels are much larger than the others."""
    gain = torch.randn((shape[1],), generator=gen, device="cuda").mul_(0.5).exp_()
    return torch.randn(shape, generator=gen, device="cuda").mul_(gain).to(torch.bfloat16)


def _grads(shape, gen):
    """Gradients: small, each row of a size of its own."""
    size = torch.randn((shape[0], 1), generator=gen, device="cuda").exp_().mul_(1e-3)
    return torch.randn(shape, generator=gen, device="cuda").mul_(size).to(torch.bfloat16)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    if op in ("norm", "norm_grad"):
        rows, H = case["rows"], case["H"]
        s = dict(op=op, rows=rows, H=H, center=case["center"], eps=1e-6)
        x = torch.randn((rows, H), generator=gen, device="cuda")
        x.mul_(torch.randn((H,), generator=gen, device="cuda").mul_(0.5).exp_())
        x.mul_(torch.randn((rows, 1), generator=gen, device="cuda").mul_(0.7).exp_())
        if case["center"]:
            x.add_(torch.randn((rows, 1), generator=gen, device="cuda"))
        s["x"] = x if case["x"] == "f32" else x.to(torch.bfloat16)
        s["weight"] = torch.randn((H,), generator=gen, device="cuda").mul_(0.1).add_(1.0)
        s["bias"] = torch.randn((H,), generator=gen, device="cuda").mul_(0.1) if case["center"] else None
        if op == "norm":
            s["out"] = torch.empty((rows, H), dtype=torch.bfloat16, device="cuda")
        else:
            # the forward pass keeps each row's mean and 1 / sqrt(var + eps)
            s["stats"] = torch.stack(_row_stats(s["x"].float(), s["center"], s["eps"]), dim=1).contiguous()
            s["dy"] = _grads((rows, H), gen)
            s["dx"] = torch.empty_like(s["x"])
            s["dweight"] = torch.empty((H,), device="cuda")
            s["dbias"] = torch.empty((H,), device="cuda") if case["center"] else None
        return s
    T, k, E = case["T"], case["k"], case["E"]
    P = T * k
    # each token's k experts: noise and a preference of the experts
    liking = torch.randn((E,), generator=gen, device="cuda") * case["skew"]
    ids = (torch.randn((T, E), generator=gen, device="cuda") + liking).topk(k, dim=1).indices
    pairs = ids.reshape(-1).sort(stable=True).indices.to(torch.int32)
    counts = torch.bincount(ids.reshape(-1), minlength=E)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = counts.cumsum(0)
    s = dict(op=op, T=T, k=k, E=E, offsets=offsets, counts=counts.tolist(), pairs=pairs, tokens=pairs.long() // k)
    if op in ("ffn", "ffn_grad"):
        H, I = case["H"], case["I"]
        s.update(H=H, I=I, x=_acts((T, H), gen))
        for name, N, K in (("gate", I, H), ("up", I, H), ("down", H, I)):
            s["q_" + name], s["s_" + name] = _stack(E, N, K, gen)
        if op == "ffn":
            s["y"] = torch.empty((P, H), dtype=torch.bfloat16, device="cuda")
        else:
            s["dy"] = _grads((P, H), gen)
            s["dx"] = torch.empty((P, H), dtype=torch.bfloat16, device="cuda")
            for name, N, K in (("gate", I, H), ("up", I, H), ("down", H, I)):
                s["dw_" + name] = torch.empty((E, N, K), dtype=torch.bfloat16, device="cuda")
        return s
    N, K = case["N"], case["K"]
    s.update(N=N, K=K)
    if k == 1:
        s["pairs"] = s["tokens"] = None  # rows already in sorted order
    s["a" if op == "product" else "dout"] = _acts((T, K), gen) if op == "product" else _grads((P, N), gen)
    s["q_w"], s["s_w"] = _stack(E, N, K, gen)
    s["out"] = torch.empty((P, N if op == "product" else K), dtype=torch.bfloat16, device="cuda")
    return s


# ---- the framework's calls ----


def _scratch(s, moe):
    """What a program keeps from call to call: the shape, codes, workspace."""
    if s["op"] in ("product", "input_grad"):
        rows, width = (s["T"], s["K"]) if s["op"] == "product" else (s["T"] * s["k"], s["N"])
        s["codes"] = torch.empty((rows, width), dtype=torch.float8_e4m3fn, device="cuda")
        s["scales"] = torch.empty((rows, moe.moe_fp8_block_scales(width)), dtype=torch.uint8, device="cuda")
        s["problem"] = moe.MoEGemmProblem(s["T"] * s["k"], s["T"], s["E"], s["N"], s["K"], s["k"])
        need = moe.moe_gemm_workspace_bytes(s["problem"])
    elif s["op"] in ("ffn", "ffn_grad"):
        s["problem"] = moe.MoEProblem(s["T"], s["H"], s["I"], s["E"], 1, 1, s["k"], 1.0)
        size = moe.moe_fp8_block_workspace_bytes if s["op"] == "ffn" else moe.moe_fp8_block_backward_workspace_bytes
        need = size(s["problem"])
    else:
        need = moe.moe_norm_workspace_bytes(s["rows"], s["H"]) if s["op"] == "norm_grad" else 0
    s["ws"] = torch.empty(max(16, need), dtype=torch.uint8, device="cuda")


def _own(s):
    from group_limited_routing_router_amd import moe

    if "ws" not in s:
        _scratch(s, moe)
    if s["op"] == "product":
        moe.moe_quantize_rows_fp8_block(s["a"], s["codes"], s["scales"])
        moe.moe_grouped_gemm_fp8_block(s["problem"], s["codes"], s["scales"], s["pairs"], s["offsets"], s["q_w"], s["s_w"], s["out"], s["ws"])
        return s["out"]
    if s["op"] == "input_grad":
        moe.moe_quantize_rows_fp8_block(s["dout"], s["codes"], s["scales"])
        moe.moe_grouped_gemm_fp8_block_dgrad(s["problem"], s["codes"], s["scales"], s["offsets"], s["q_w"], s["s_w"], s["out"], s["ws"])
        return s["out"]
    if s["op"] == "norm":
        moe.moe_norm(s["x"], s["weight"], s["bias"], s["eps"], s["out"], center=s["center"])
        return s["out"]
    if s["op"] == "norm_grad":
        moe.moe_norm_backward(s["dy"], s["x"], s["weight"], s["stats"], s["dx"], s["dweight"], s["dbias"], s["ws"], center=s["center"])
        return s["dx"], s["dweight"], s["dbias"]
    weights = [s[p + n] for n in ("gate", "up", "down") for p in ("q_", "s_")]
    if s["op"] == "ffn":
        moe.moe_expert_ffn_fp8_block(s["problem"], s["x"], s["pairs"], s["offsets"], *weights, s["y"], s["ws"])
        return s["y"]
    moe.moe_expert_ffn_fp8_block_backward(s["problem"], s["x"], s["pairs"], s["offsets"], *weights, s["dy"], s["dx"],
                                          s["dw_gate"], s["dw_up"], s["dw_down"], s["ws"])
    return s["dx"], s["dw_gate"], s["dw_up"], s["dw_down"]


# ---- the plain form ----


def _row_stats(x, center, eps):
    mean = x.mean(dim=1) if center else torch.zeros_like(x[:, 0])
    var = (x - mean[:, None]).square().mean(dim=1)
    return mean, 1.0 / torch.sqrt(var + eps)


def _plain_norm(s):
    x = s["x"].float()
    if s["op"] == "norm":
        mean, r = _row_stats(x, s["center"], s["eps"])
        y = (x - mean[:, None]) * r[:, None] * s["weight"]
        return (y if s["bias"] is None else y + s["bias"]).to(torch.bfloat16)
    mean, r = s["stats"][:, :1], s["stats"][:, 1:]
    xh, dy = (x - mean) * r, s["dy"].float()
    g = dy * s["weight"]
    off = (g * xh).mean(dim=1, keepdim=True) * xh
    if s["center"]:
        off = off + g.mean(dim=1, keepdim=True)
    return ((g - off) * r).to(s["x"].dtype), (dy * xh).sum(dim=0), dy.sum(dim=0) if s["center"] else None


def _by_expert(s, x):
    """The rows of each expert, from rows in sorted order."""
    return x.split(s["counts"])


def _plain_ffn_grad(s):
    """Expert by expert, so that nothing large is held in fp32."""
    x, xr = s["x"], _rounded_rows(s["x"].float())

    def expert(e, tokens, dy):
        a, wg, wu, wd = xr[tokens], _weights(s, "gate", e), _weights(s, "up", e), _weights(s, "down", e)
        g, u, dh = a @ wg.t(), a @ wu.t(), _rounded_rows(dy.float()) @ wd
        sg = 1.0 / (1.0 + torch.exp(-g))
        h, dg, du = g * sg * u, dh * u * sg * (1.0 + g * (1.0 - sg)), dh * g * sg
        dx = _rounded_rows(dg) @ wg + _rounded_rows(du) @ wu
        rows = x[tokens].float()
        dws = [(l.bfloat16().float().t() @ r.bfloat16().float()).bfloat16() for l, r in ((dg, rows), (du, rows), (dy, h))]
        return [dx.bfloat16(), *dws]

    parts = [expert(e, t, d) for e, (t, d) in enumerate(zip(_by_expert(s, s["tokens"]), _by_expert(s, s["dy"])))]
    dx, *dws = zip(*parts)
    return (torch.cat(dx), *(torch.stack(d) for d in dws))


def _plain(s):
    op = s["op"]
    if op in ("norm", "norm_grad"):
        return _plain_norm(s)
    if op == "ffn_grad":
        return _plain_ffn_grad(s)
    if op == "ffn":
        xr = _rounded_rows(s["x"].float())

        def expert(e, a):
            g, u = a @ _weights(s, "gate", e).t(), a @ _weights(s, "up", e).t()
            h = g / (1.0 + torch.exp(-g)) * u
            return (_rounded_rows(h) @ _weights(s, "down", e).t()).bfloat16()

        return torch.cat([expert(e, xr[t]) for e, t in enumerate(_by_expert(s, s["tokens"]))])
    rows = _rounded_rows((s["a"] if op == "product" else s["dout"]).float())
    if op == "product" and s["tokens"] is not None:
        rows = rows[s["tokens"]]
    parts = [r @ (_weights(s, "w", e).t() if op == "product" else _weights(s, "w", e)) for e, r in enumerate(_by_expert(s, rows))]
    return torch.cat(parts).to(s["out"].dtype)


def run(state):
    return _own(state) if own else _plain(state)


# ---- what a pass cannot do without ----


def work(case):
    if case["op"] in ("norm", "norm_grad"):
        n, size = case["rows"] * case["H"], 4 if case["x"] == "f32" else 2
        if case["op"] == "norm":
            return {"bytes": n * (size + 2) + 4 * case["H"] * (1 + case["center"]), "flops": 6.0 * n}
        return {"bytes": n * (size + 2 + size) + 8 * case["rows"] + 4 * case["H"] * (2 + case["center"]), "flops": 12.0 * n}
    T, k, E = case["T"], case["k"], case["E"]
    P = T * k
    met = E * (1.0 - (1.0 - 1.0 / E) ** P) if E > 1 else 1.0  # experts with rows, in the mean over routings
    index = 4 * (E + 1) + (4 * P if k > 1 else 0)
    if case["op"] in ("ffn", "ffn_grad"):
        H, I = case["H"], case["I"]
        if case["op"] == "ffn":
            return {"bytes": 2 * T * H + 3 * met * H * I + 2 * P * H + index, "flops": 6.0 * P * H * I}
        return {"bytes": 2 * T * H + 2 * P * H + 3 * met * H * I + 2 * P * H + 6 * E * H * I + index, "flops": 16.0 * P * H * I}
    N, K = case["N"], case["K"]
    read, written = (T * K, P * N) if case["op"] == "product" else (P * N, P * K)
    return {"bytes": 2 * read + met * N * K + 2 * written + index, "flops": 2.0 * P * N * K}


# ---- the definition in 64 bits ----


def _scale64(top):
    """The scale of blocks whose largest magnitude is top: doubled until top fits."""
    s = torch.exp2(torch.floor(torch.log2(torch.where(top > 0, top, torch.ones_like(top)) / 448)))
    s = torch.where(top / s > 448, 2 * s, s)
    s = torch.where(top / s <= 224, s / 2, s)
    return torch.where(top > 0, s, torch.ones_like(s))


def _round64(x):
    """x to the nearest e4m3: 4 significant bits, steps of 2^-9 at the least."""
    size = torch.floor(torch.log2(torch.clamp(x.abs(), min=2.0 ** -6)))
    step = torch.exp2(size - 3)
    return torch.round(x / step) * step


def _rows64(x):
    got = torch.empty_like(x, dtype=torch.float64)
    for c in range(0, x.shape[1], BLOCK):
        part = x[:, c:c + BLOCK].double()
        s = _scale64(part.abs().max(dim=1, keepdim=True).values) if part.numel() else 1.0
        got[:, c:c + BLOCK] = _round64(part / s) * s
    return got


def _weights64(s, name, e):
    w = s["q_" + name][e].double()
    factor = torch.exp2(s["s_" + name][e].double() - 127)
    for i in range(factor.shape[0]):
        w[i * BLOCK:(i + 1) * BLOCK] *= factor[i].repeat_interleave(BLOCK)[: w.shape[1]]
    return w


def _norm64(s):
    x, w = s["x"].double(), s["weight"].double()
    if s["op"] == "norm":
        mean = x.sum(dim=1, keepdim=True) / s["H"] if s["center"] else 0.0
        y = (x - mean) / ((((x - mean) ** 2).sum(dim=1, keepdim=True)) / s["H"] + s["eps"]).sqrt() * w
        return y if s["bias"] is None else y + s["bias"].double()
    dy, r = s["dy"].double(), s["stats"][:, 1:].double()
    xh = (x - s["stats"][:, :1].double()) * r
    g = dy * w
    dx = g - xh * ((g * xh).sum(dim=1, keepdim=True) / s["H"])
    if s["center"]:
        dx = dx - g.sum(dim=1, keepdim=True) / s["H"]
    return dx * r, (dy * xh).sum(dim=0), dy.sum(dim=0) if s["center"] else None


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("norm", "norm_grad"):
        return _norm64(s)
    P, E = case["T"] * case["k"], case["E"]
    bounds = s["offsets"].tolist()
    row = s["tokens"] if s["tokens"] is not None else torch.arange(P, device="cuda")
    empty = lambda *shape: torch.zeros(shape, dtype=torch.float64, device="cuda")  # noqa: E731
    if op in ("product", "input_grad"):
        rows = _rows64(s["a"] if op == "product" else s["dout"])
        got = empty(*s["out"].shape)
    else:
        xr = _rows64(s["x"])
        got = empty(P, case["H"])
        grads = {n: empty(*s["dw_" + n].shape) for n in ("gate", "up", "down")} if op == "ffn_grad" else {}
    for e in range(E):
        i, j = bounds[e], bounds[e + 1]
        if i == j:
            continue
        if op == "product":
            got[i:j] = rows[row[i:j]] @ _weights64(s, "w", e).t()
            continue
        if op == "input_grad":
            got[i:j] = rows[i:j] @ _weights64(s, "w", e)
            continue
        wg, wu, wd = (_weights64(s, n, e) for n in ("gate", "up", "down"))
        g, u = xr[row[i:j]] @ wg.t(), xr[row[i:j]] @ wu.t()
        sig = torch.sigmoid(g)
        h = g * sig * u
        if op == "ffn":
            got[i:j] = _rows64(h) @ wd.t()
            continue
        dh = _rows64(s["dy"][i:j]) @ wd
        dg, du = dh * u * (sig + g * sig * (1 - sig)), dh * g * sig
        got[i:j] = _rows64(dg) @ wg + _rows64(du) @ wu
        x = s["x"][row[i:j]].double()
        for name, left, right in (("gate", dg, x), ("up", du, x), ("down", s["dy"][i:j], h)):
            torch.mm(left.to(torch.bfloat16).double().t(), right.to(torch.bfloat16).double(), out=grads[name][e])
    return (got, grads["gate"], grads["up"], grads["down"]) if op == "ffn_grad" else got
