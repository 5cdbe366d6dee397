"""The grouped products (include/moe_gemm.h) against 64-bit references, with
tolerances counted from the additions and roundings (tests/_grouped.py); the
int8 product and the row quantisation bit for bit.  Outputs start as NaN, and
rows that belong to no expert have to keep it, with NaN in the inputs there."""
import numpy as np
import pytest
import torch

from _grouped import Case, problem, tolerance, worst

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    from group_limited_routing_router_amd import moe as m
    m.load_library()
    return m


def dev(t):
    return None if t is None else t.cuda()


def ws_for(moe, g):
    n = moe.moe_gemm_workspace_bytes(g)
    return torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda") if n else None


def run(moe, c, op, dtype, offsets=True, accumulate=None, stream=None):
    """One call on a case's inputs; accumulate: what the output starts as."""
    g = c.problem()
    off = dev(c.offsets) if offsets else None
    ws = ws_for(moe, g)
    shape = {"input_grad": (c.P, c.K), "weight_grad": (c.E, c.N, c.K)}.get(op, (c.P, c.N))
    out = (torch.full(shape, float("nan"), dtype=dtype, device="cuda") if accumulate is None
           else accumulate.clone())
    acc = accumulate is not None
    if op == "product":
        moe.moe_grouped_gemm(g, dev(c.a), dev(c.pairs), off, dev(c.w), out, ws, stream=stream)
    elif op == "input_grad":
        moe.moe_grouped_gemm_dgrad(g, dev(c.dout), off, dev(c.w), out, ws, accumulate=acc, stream=stream)
    elif op == "weight_grad":
        moe.moe_grouped_gemm_wgrad(g, dev(c.dout), dev(c.a), dev(c.pairs), off, out, ws,
                                   accumulate=acc, stream=stream)
    else:
        moe.moe_grouped_gemm_int8(g, dev(c.a8), dev(c.a_scale), dev(c.pairs), off, dev(c.w8),
                                  dev(c.w_scale), out, ws, stream=stream)
    torch.cuda.synchronize()
    return out.cpu()


def check(c, op, dtype, got, start=None):
    own = c.owned()
    got = got.to(c.a.device)
    own = own.to(c.a.device)
    if op == "int8":
        ref = c.int8().to(dtype)
        assert torch.equal(got[own], ref[own]), f"{int((got[own] != ref[own]).sum())} values differ"
    else:
        ref, mag, length = getattr(c, op)()
        if start is not None:
            ref = ref + start.double()
        tol = tolerance(ref, mag, length, dtype, start)
        if op == "weight_grad":
            own = torch.ones(c.E, dtype=torch.bool, device=got.device)
        w = worst(got[own], ref[own], tol[own])
        assert w <= 1.0, f"error {w:.3g} of the tolerance"
    if op != "weight_grad" and start is None:
        assert bool(torch.isnan(got[~own].float()).all()), "a row of no expert was written"


SHAPES = [
    # P, E, N, K, k, kind
    (1, 1, 64, 64, 1, "even"),          # one token, one group
    (1, 4, 16, 16, 1, "random"),        # the smallest products
    (3, 5, 80, 48, 1, "random"),
    (7, 3, 208, 144, 2, "random"),
    (16, 1, 512, 1024, 1, "even"),
    (33, 2, 272, 336, 4, "one"),
    (64, 16, 128, 256, 4, "random"),
    (100, 7, 336, 80, 2, "even"),
    (257, 3, 256, 256, 1, "even"),
    (300, 256, 64, 128, 8, "random"),   # more experts than rows for most
    (513, 2, 528, 512, 1, "one"),
    (600, 5, 304, 784, 3, "random"),
    (1031, 9, 1008, 272, 1, "random"),
    (2100, 4, 256, 640, 6, "random"),
    (5, 1, 128, 4112, 1, "even"),       # split reductions: the product's
    (40, 2, 192, 2064, 2, "random"),
    (3, 1, 2064, 128, 1, "even"),       # ... the input gradient's
    (4400, 3, 4112, 144, 1, "random"),
    (4400, 3, 160, 4112, 2, "random"),
    (70, 2, 3088, 144, 1, "random"),
    (2500, 2, 144, 176, 1, "random"),   # ... the weight gradient's
    (1700, 1, 64, 80, 2, "even"),
]
IDS = ["P%d_E%d_N%d_K%d_k%d_%s" % s for s in SHAPES]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("op", ["product", "input_grad", "weight_grad", "int8"])
@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_against_64_bits(moe, shape, op, dtype):
    P, E, N, K, k, kind = shape
    print(f"[case] {op} {shape} {dtype}", flush=True)
    c = Case(P, E, N, K, k, kind, seed=P + N)
    check(c, op, dtype, run(moe, c, op, dtype))


@pytest.mark.parametrize("op", ["product", "input_grad", "weight_grad", "int8"])
@pytest.mark.parametrize("shape,dtype", [
    ((9000, 8, 4096, 1008, 1), torch.bfloat16),   # many tiles: 256 rows each
    ((4500, 8, 1008, 4096, 2), torch.float32),
    ((1000, 256, 1040, 1024, 4), torch.bfloat16),  # a large weight stream and few rows
    ((7000, 256, 1040, 1024, 1), torch.float32),
    ((12000, 256, 1040, 1024, 8), torch.bfloat16),
    ((60, 64, 520, 648, 2), torch.bfloat16),      # most experts idle
    ((100, 37, 520, 648, 1), torch.float32),
], ids=lambda s: "P%d_E%d_N%d_K%d_k%d" % s if isinstance(s, tuple) else str(s).split(".")[1])
def test_large(moe, shape, dtype, op):
    """The tiles and weight streams of larger shapes (references on the GPU)."""
    print(f"[case] {op} {shape} {dtype}", flush=True)
    if op == "int8" and shape[3] % 16:
        shape = (*shape[:3], shape[3] // 16 * 16, shape[4])
    c = Case(*shape, kind="random", seed=shape[0], first=3, behind=9, device="cuda")
    check(c, op, dtype, run(moe, c, op, dtype))


@pytest.mark.parametrize("op", ["product", "input_grad", "weight_grad"])
@pytest.mark.parametrize("shape", [(45, 3, 40, 24, 1), (130, 4, 8, 136, 2), (77, 2, 264, 8, 1),
                                   (400, 3, 312, 328, 2)],
                         ids=lambda s: "P%d_E%d_N%d_K%d_k%d" % s)
def test_multiples_of_eight(moe, shape, op):
    print(f"[case] {op} {shape}", flush=True)
    c = Case(*shape, kind="random", seed=5)
    check(c, op, torch.float32, run(moe, c, op, torch.float32))


@pytest.mark.parametrize("op", ["product", "input_grad", "weight_grad", "int8"])
@pytest.mark.parametrize("shape", [(90, 4, 64, 96, 1), (500, 3, 272, 320, 2), (40, 1, 512, 512, 1),
                                   (40, 2, 96, 2064, 1), (40, 2, 2064, 96, 2), (1500, 1, 80, 96, 2)],
                         ids=lambda s: "P%d_E%d_N%d_K%d_k%d" % s)
def test_rows_of_no_expert(moe, shape, op):
    """Positions before the first expert's and behind the last's: not read
    (NaN there) and not written."""
    print(f"[case] {op} {shape}", flush=True)
    c = Case(*shape, kind="random", seed=9, first=5, behind=11)
    own = c.owned()
    c.dout[~own] = float("nan")
    used = torch.zeros(c.S, dtype=torch.bool)
    used[c.rows[own]] = True
    c.a[~used] = float("nan")
    c.a_scale[~used] = float("nan")
    check(c, op, torch.float32, run(moe, c, op, torch.float32))


@pytest.mark.parametrize("op", ["product", "input_grad", "weight_grad", "int8"])
@pytest.mark.parametrize("P,N,K", [(1, 512, 512), (5, 272, 128), (300, 128, 528)])
def test_one_group_without_offsets(moe, op, P, N, K):
    print(f"[case] {op} P={P} N={N} K={K}", flush=True)
    c = Case(P, 1, N, K, kind="even", seed=3)
    check(c, op, torch.float32, run(moe, c, op, torch.float32, offsets=False))


@pytest.mark.parametrize("op", ["input_grad", "weight_grad"])
@pytest.mark.parametrize("shape", [(60, 4, 72, 40, 1), (700, 3, 272, 320, 2), (9, 1, 640, 768, 1),
                                   (6, 1, 2056, 72, 1), (1500, 1, 72, 80, 2), (4500, 8, 1008, 4096, 2)],
                         ids=lambda s: "P%d_E%d_N%d_K%d_k%d" % s)
def test_accumulate(moe, op, shape):
    print(f"[case] {op} {shape}", flush=True)
    c = Case(*shape, kind="random", seed=8, device="cuda")
    out = (c.P, c.K) if op == "input_grad" else (c.E, c.N, c.K)
    start = torch.randn(out, generator=torch.Generator().manual_seed(1)).cuda()
    check(c, op, torch.float32, run(moe, c, op, torch.float32, accumulate=start), start)


def test_weight_gradient_without_rows(moe):
    """No positions at all: zeros, or what accumulate finds."""
    g = problem(0, 0, 3, 40, 24)
    dw = torch.full((3, 40, 24), float("nan"), device="cuda")
    off = torch.zeros(4, dtype=torch.int32, device="cuda")
    ws = ws_for(moe, g)
    moe.moe_grouped_gemm_wgrad(g, None, None, None, off, dw, ws)
    torch.cuda.synchronize()
    assert bool((dw == 0).all())
    dw.fill_(3.0)
    moe.moe_grouped_gemm_wgrad(g, None, None, None, off, dw, ws, accumulate=True)
    torch.cuda.synchronize()
    assert bool((dw == 3.0).all())


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("P,E,N,K", [(30, 3, 64, 64), (700, 3, 272, 320)])
def test_one_bad_row_stays_alone(moe, P, E, N, K, bad):
    """A NaN or infinity in one activation or gradient row reaches its own
    output row, and in the weight gradient its own expert's, alone."""
    c = Case(P, E, N, K, kind="even", seed=4)
    q = P // 2
    e = next(e for e, i, j in c.spans() if i <= q < j)
    good = {op: run(moe, c, op, torch.float32) for op in ("product", "input_grad", "weight_grad")}
    c.a[q, 3] = bad
    c.dout[q, 5] = bad
    for op in ("product", "input_grad"):
        got = run(moe, c, op, torch.float32)
        keep = torch.arange(P) != q
        assert torch.equal(got[keep], good[op][keep]), op
        assert not bool(torch.isfinite(got[q]).any()), op
    got = run(moe, c, "weight_grad", torch.float32)
    keep = torch.arange(E) != e
    assert torch.equal(got[keep], good["weight_grad"][keep])
    assert not bool(torch.isfinite(got[e][5]).any()) and not bool(torch.isfinite(got[e][:, 3]).any())


def test_wrong_indices_stay_in_range(moe):
    """Offsets and pairs out of range are clamped: nothing out of range is
    read or written (the rows around the output keep their values)."""
    c = Case(64, 4, 64, 64, 2, "even", seed=6)
    c.pairs[::3] = 1 << 30
    c.pairs[1::3] = -5
    c.rows = (c.pairs.long() // 2).clamp(0, c.S - 1)
    c.rows[c.pairs < 0] = 0
    check(c, "product", torch.float32, run(moe, c, "product", torch.float32))
    check(c, "weight_grad", torch.float32, run(moe, c, "weight_grad", torch.float32))
    c.offsets[-1] = 1 << 30
    c.offsets[0] = -7
    g = c.problem()
    out = torch.full((c.P + 2, c.N), 7.0, device="cuda")
    moe.moe_grouped_gemm(g, dev(c.a), dev(c.pairs), dev(c.offsets), dev(c.w), out[1:-1], ws_for(moe, g))
    torch.cuda.synchronize()
    assert bool((out[0] == 7).all()) and bool((out[-1] == 7).all())


def quantize_ref(x):
    xf = x.double()
    amax = xf.abs().amax(dim=1)
    bad = ~torch.isfinite(xf).all(dim=1)
    zero = bad | (amax < 2.0 ** -100)
    codes = torch.round(127 * xf / torch.where(zero, 1.0, amax)[:, None])
    codes[zero] = 0
    scale = torch.where(zero, torch.ones(len(x)), (amax.float() / 127.0))
    scale[bad] = float("nan")
    return codes.to(torch.int8), scale


@pytest.mark.parametrize("rows,K", [(1, 16), (3, 48), (17, 256), (130, 2064), (5, 5120), (2, 65536),
                                    (4099, 128), (2100, 1040), (20, 16384), (19, 8208)])
def test_quantize_rows(moe, rows, K):
    print(f"[case] quantize {rows} x {K}", flush=True)
    gen = torch.Generator().manual_seed(rows + K)
    x = torch.randn((rows, K), generator=gen) * torch.exp(3 * torch.randn((rows, 1), generator=gen))
    x = x.to(torch.bfloat16)
    x[0, : K // 2] = x[0].abs().max() / 2     # quotients half way between two codes
    if rows > 16:
        x[1] = 0
        x[2, 5] = float("nan")
        x[3, 7] = float("inf")
        x[4] = 3e38 * torch.sign(x[4].float()).to(torch.bfloat16)
        x[5] = x[5] * 2.0 ** -120
        x[6] = -0.0
        x[7, 1:] = 0
        x[8] = torch.arange(K).to(torch.bfloat16) - K // 2
    codes = torch.full((rows + 1, K), 99, dtype=torch.int8, device="cuda")
    scales = torch.full((rows + 1,), 9.0, device="cuda")
    moe.moe_quantize_rows_int8(x.cuda(), codes, scales)
    torch.cuda.synchronize()
    rc, rs = quantize_ref(x)
    assert torch.equal(codes[:rows].cpu(), rc)
    assert torch.equal(scales[:rows].cpu().nan_to_num(nan=-1.0), rs.nan_to_num(nan=-1.0))
    assert bool((codes[rows] == 99).all()) and float(scales[rows]) == 9.0
