"""Cases of the experts' matrix products: by expert with ragged sizes, with
their two gradients, and in 8-bit integers with a scale for each token and
each output channel.

Positions q of the products are sorted by expert: expert e owns the positions
offsets[e] .. offsets[e + 1].  With k > 1, position q belongs to token
sorted_pairs[q] // k and the activations are gathered by it; with k = 1 the
rows are already in sorted order.

    product      out[q] = a[row(q)] . w[e]^T
    input_grad   da[q]  = dout[q] . w[e]
    weight_grad  dw[e]  = sum over e's q of dout[q]^T a[row(q)]
    int8         a is quantised by rows (scale s_a = amax / 127, codes
                 127 a / amax to the nearest, ties to even),
                 out[q] = s_a[row(q)] s_w[e] (codes . codes^T)

a [T, K], w [E, N, K] and dout [T k, N] are bf16 (the weights of the int8
product are int8 codes with fp32 scales [E, N]); out is fp32 or bf16.
"""
import math

import torch

own = False

# one weight matrix of the repository's block: hidden 5120, intermediate 2560,
# 256 experts, 8 for each token
HIDDEN, INTER, EXPERTS, TOP = 5120, 2560, 256, 8


def listed():
    block = dict(E=EXPERTS, k=TOP, skew=0.0)
    return [
        # the smallest configuration's gate projection: a launch's latency
        dict(name="product tiny", op="product", T=64, k=4, E=16, N=128, K=256, out="bf16", skew=0.0),
        # a decode batch: 4 rows for each expert, every weight read once
        dict(name="product decode", op="product", T=128, N=INTER, K=HIDDEN, out="bf16", **block),
        # a prefill chunk: 256 rows for each expert
        dict(name="product prefill", op="product", T=8192, N=INTER, K=HIDDEN, out="bf16", **block),
        # the gradient of the down projection's input, busy and idle experts
        dict(name="input_grad skewed", op="input_grad", T=4096, k=TOP, E=EXPERTS, N=HIDDEN, K=INTER, out="bf16", skew=0.7),
        # few experts, odd sizes, rows in sorted order
        dict(name="input_grad odd", op="input_grad", T=5003, k=1, E=24, N=1000, K=776, out="f32", skew=0.5),
        # the gradient of the gate projection in a training step
        dict(name="weight_grad chunk", op="weight_grad", T=8192, N=INTER, K=HIDDEN, out="bf16", **block),
        # odd sizes, one expert may be left without a row; fp32 for the optimiser
        dict(name="weight_grad odd", op="weight_grad", T=1501, k=3, E=24, N=776, K=1000, out="f32", skew=1.0),
        # a dense layer's product for one token (one group that takes every row)
        dict(name="int8 one token", op="int8", T=1, k=1, E=1, N=20480, K=HIDDEN, out="bf16", skew=0.0),
        dict(name="int8 decode", op="int8", T=128, N=INTER, K=HIDDEN, out="bf16", **block),
        dict(name="int8 prefill", op="int8", T=8192, N=INTER, K=HIDDEN, out="bf16", **block),
        dict(name="int8 odd", op="int8", T=301, k=2, E=8, N=1208, K=2000, out="f32", skew=0.3),
        # a dense layer over a whole prefill chunk
        dict(name="product dense", op="product", T=8192, k=1, E=1, N=HIDDEN, K=20480, out="f32", skew=0.0),
    ]


def _between(rng, low, high, step=1):
    """A whole number of [low, high], even over its logarithm, a multiple of step."""
    return max(low, int(math.exp(rng.uniform(math.log(low), math.log(high + 1)))) // step * step)


def draw(rng):
    op = rng.choice(["product", "input_grad", "weight_grad", "int8"])
    step = 16 if op == "int8" else 8
    E = _between(rng, 1, EXPERTS)
    k = 1 if op == "input_grad" else min(E, rng.choice([1, 1, 2, 4, 8]))
    N, K = (_between(rng, 64, 20480, step) for _ in range(2))
    while E * N * K > EXPERTS * INTER * HIDDEN:
        N, K = max(64, N // 2 // step * step), max(64, K // 2 // step * step)
    T = _between(rng, 1, 65536 // k)
    while T * k * N * K > 8192 * TOP * INTER * HIDDEN:
        T = max(1, T // 2)
    return dict(op=op, T=T, k=k, E=E, N=N, K=K, out=rng.choice(["f32", "bf16"]),
                skew=rng.choice([0.0, 0.3, 0.7, 1.0]))


def _randn(shape, gen, scale):
    """bf16 normal values; the large stacks are drawn a slice at a time."""
    x = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
    part = max(1, (1 << 28) // max(1, x[0].numel()))
    for s in range(0, shape[0], part):
        n = min(part, shape[0] - s)
        x[s:s + n] = torch.randn((n, *shape[1:]), generator=gen, device="cuda").mul_(scale)
    return x


def prepare(case, seed):
    T, k, E, N, K = (case[x] for x in ("T", "k", "E", "N", "K"))
    gen = torch.Generator(device="cuda").manual_seed(seed)
    P = T * k
    # each token's k experts: noise and a preference of the experts
    liking = torch.randn((E,), generator=gen, device="cuda") * case["skew"]
    ids = (torch.randn((T, E), generator=gen, device="cuda") + liking).topk(k, dim=1).indices
    sorted_pairs = ids.reshape(-1).sort(stable=True).indices.to(torch.int32)
    counts = torch.bincount(ids.reshape(-1), minlength=E)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = counts.cumsum(0)
    s = dict(op=case["op"], T=T, k=k, E=E, N=N, K=K, offsets=offsets, counts=counts.tolist(),
             pairs=sorted_pairs if k > 1 else None,
             tokens=sorted_pairs.long() // k if k > 1 else None)
    if case["op"] != "input_grad":
        # activations: a few channels are much larger than the others
        gain = torch.randn((K,), generator=gen, device="cuda").mul_(0.5).exp_()
        s["a"] = (_randn((T, K), gen, 1.0) * gain).to(torch.bfloat16)
    if case["op"] in ("input_grad", "weight_grad"):
        # gradients: small, each row of a size of its own
        size = torch.randn((P, 1), generator=gen, device="cuda").exp_().mul_(1e-3)
        s["dout"] = (_randn((P, N), gen, 1.0) * size).to(torch.bfloat16)
    if case["op"] in ("product", "input_grad"):
        s["w"] = _randn((E, N, K), gen, 0.02)
    if case["op"] == "int8":
        w = torch.empty((E, N, K), dtype=torch.int8, device="cuda")
        for e in range(E):
            w[e].copy_(torch.randn((N, K), generator=gen, device="cuda").mul_(32.0).round_().clamp_(-127, 127))
        s["w"] = w
        s["w_scale"] = torch.rand((E, N), generator=gen, device="cuda").mul_(4e-4).add_(4e-4)
    shape = {"input_grad": (P, K), "weight_grad": (E, N, K)}.get(case["op"], (P, N))
    s["out"] = torch.empty(shape, dtype=torch.float32 if case["out"] == "f32" else torch.bfloat16, device="cuda")
    return s


def _own(s):
    from group_limited_routing_router_amd import moe

    if "problem" not in s:
        # a program keeps its workspace from call to call
        s["problem"] = moe.MoEGemmProblem(s["T"] * s["k"], s["T"], s["E"], s["N"], s["K"], s["k"])
        s["ws"] = torch.empty(max(16, moe.moe_gemm_workspace_bytes(s["problem"])), dtype=torch.uint8, device="cuda")
        if s["op"] == "int8":
            s["codes"] = torch.empty((s["T"], s["K"]), dtype=torch.int8, device="cuda")
            s["a_scale"] = torch.empty((s["T"],), dtype=torch.float32, device="cuda")
    g, out = s["problem"], s["out"]
    if s["op"] == "product":
        moe.moe_grouped_gemm(g, s["a"], s["pairs"], s["offsets"], s["w"], out, s["ws"])
    elif s["op"] == "input_grad":
        moe.moe_grouped_gemm_dgrad(g, s["dout"], s["offsets"], s["w"], out, s["ws"])
    elif s["op"] == "weight_grad":
        moe.moe_grouped_gemm_wgrad(g, s["dout"], s["a"], s["pairs"], s["offsets"], out, s["ws"])
    else:
        moe.moe_quantize_rows_int8(s["a"], s["codes"], s["a_scale"])
        moe.moe_grouped_gemm_int8(g, s["codes"], s["a_scale"], s["pairs"], s["offsets"], s["w"], s["w_scale"], out, s["ws"])
    return out


def _rows(s, x):
    """The sorted rows of the activations x."""
    return x if s["tokens"] is None else x[s["tokens"]]


def _plain(s):
    out, counts = s["out"], s["counts"]
    if s["op"] == "weight_grad":
        x = _rows(s, s["a"])
        return torch.stack([(d.float().t() @ r.float()).to(out.dtype) for d, r in
                            zip(s["dout"].split(counts), x.split(counts))])
    if s["op"] == "product":
        parts = [r.float() @ w.float().t() for r, w in zip(_rows(s, s["a"]).split(counts), s["w"])]
    elif s["op"] == "input_grad":
        parts = [d.float() @ w.float() for d, w in zip(s["dout"].split(counts), s["w"])]
    else:
        a = s["a"].float()
        amax = a.abs().amax(dim=1, keepdim=True)
        # 127 a is exact in 32 bits, so a quotient half way between two codes is met exactly
        codes = torch.where(amax > 0, torch.round(a * 127.0 / amax), 0.0)
        scale = torch.where(amax > 0, amax / 127.0, 1.0)
        parts = [(r @ w.float().t()) * (t * v) for r, w, t, v in
                 zip(_rows(s, codes).split(counts), s["w"], _rows(s, scale).split(counts), s["w_scale"])]
    return torch.cat(parts).to(out.dtype)


def run(state):
    return _own(state) if own else _plain(state)


def _rows_met(case):
    """The rows of the activations and the experts that a pass can meet, in the mean over routings."""
    experts = case["E"] * (1.0 - (1.0 - 1.0 / case["E"]) ** (case["T"] * case["k"])) if case["E"] > 1 else 1.0
    return case["T"], experts


def work(case):
    T, k, E, N, K = (case[x] for x in ("T", "k", "E", "N", "K"))
    P, out = T * k, 4 if case["out"] == "f32" else 2
    rows, experts = _rows_met(case)
    index = 4 * (E + 1) + (4 * P if k > 1 else 0)
    weights = experts * N * K
    bytes_ = {"product": rows * K * 2 + weights * 2 + P * N * out,
              "input_grad": P * N * 2 + weights * 2 + P * K * out,
              "weight_grad": P * N * 2 + rows * K * 2 + E * N * K * out,
              "int8": rows * K * 2 + weights + experts * N * 4 + P * N * out}[case["op"]]
    return {"bytes": bytes_ + index, "flops": 2.0 * P * N * K}


def exact(case, seed):
    s = prepare(case, seed)
    P, E, N, K = case["T"] * case["k"], case["E"], case["N"], case["K"]
    bounds = s["offsets"].tolist()
    row = s["tokens"] if s["tokens"] is not None else torch.arange(P, device="cuda")
    if case["op"] == "weight_grad":
        got = torch.zeros((E, N, K), dtype=torch.float64, device="cuda")
    else:
        got = torch.zeros((P, K if case["op"] == "input_grad" else N), dtype=torch.float64, device="cuda")
    for e in range(E):
        i, j = bounds[e], bounds[e + 1]
        if i == j:
            continue
        if case["op"] == "weight_grad":
            torch.mm(s["dout"][i:j].double().t(), s["a"][row[i:j]].double(), out=got[e])
        elif case["op"] == "input_grad":
            torch.mm(s["dout"][i:j].double(), s["w"][e].double(), out=got[i:j])
        elif case["op"] == "product":
            torch.mm(s["a"][row[i:j]].double(), s["w"][e].double().t(), out=got[i:j])
        else:
            a = s["a"][row[i:j]].double()
            top = a.abs().max(dim=1, keepdim=True).values
            codes = torch.where(top > 0, torch.round(a * 127 / top), torch.zeros_like(a))
            got[i:j] = codes @ s["w"][e].double().t() * (top / 127) * s["w_scale"][e].double()
    return got
