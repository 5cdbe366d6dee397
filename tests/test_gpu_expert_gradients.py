"""The experts' gradients against what does not use their formulas: automatic
differentiation and central differences of the forward pass, in 64 bits.

The differences are taken along the gradient's own signs, where the slope is
the sum of the gradient's magnitudes and does not cancel; a gradient of zeros
and one of the other sign have to be rejected by the same comparison."""
import pytest
import torch

from test_gpu_grouped_experts import IDS, SHAPES, backward, reference_gradients, setup

pytestmark = pytest.mark.gpu

NAMES = ("x", "w_gate", "w_up", "w_down")


@pytest.fixture(scope="module")
def moe():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    from group_limited_routing_router_amd import moe as m
    m.load_library()
    return m


def forward(q, spans, dy):
    """sum(dy y) in 64 bits; q["x"] holds a row for each sorted position."""
    total = torch.zeros((), dtype=torch.float64, device="cuda")
    for e, i, j in spans:
        x = q["x"][i:j]
        g, u = x @ q["w_gate"][e].T, x @ q["w_up"][e].T
        total = total + (dy[i:j].double() * ((g / (1 + torch.exp(-g)) * u) @ q["w_down"][e].T)).sum()
    return total


def inputs(moe, shape, seed):
    cfg, p, d, b, rows, spans = setup(moe, shape, seed)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dy = torch.randn((cfg.T * cfg.k, cfg.H), generator=gen, device="cuda").to(torch.bfloat16)
    q = {n: (d[n][rows] if n == "x" else d[n]).double() for n in NAMES}
    ref, tol = reference(cfg, d, rows, spans, dy)
    return cfg, p, d, b, spans, dy, q, ref, tol


def reference(cfg, d, rows, spans, dy):
    rdx, rdw = reference_gradients(cfg, d, rows, spans, dy)
    both = {"x": rdx, **rdw}
    return {n: both[n][0] for n in NAMES}, {n: both[n][1] for n in NAMES}


@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_reference_against_autograd(moe, shape):
    """The formulas that the kernels are tested against.  Both sides are 64-bit
    sums of at most a few thousand products: 2^-53 of each, so 2^-40 of the
    largest gradient leaves a factor of several for sums that cancel."""
    print(f"[case] autograd {shape}", flush=True)
    cfg, p, d, b, spans, dy, q, ref, _ = inputs(moe, shape, 51)
    leaves = {n: t.requires_grad_() for n, t in q.items()}
    grads = torch.autograd.grad(forward(leaves, spans, dy), [leaves[n] for n in NAMES])
    for n, g in zip(NAMES, grads):
        top = float(g.abs().max())
        assert top > 0 and float((ref[n] - g).abs().max()) <= 2.0 ** -40 * top, n


@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_gradients_along_their_signs(moe, shape):
    """The kernels' gradients along the signs of the reference's, against the
    slope there.  The tolerance is the gradients' own, summed, and 1e-5 of the
    slope for the difference (steps of 1e-6 move a gate by below 1e-3, its
    square and 2^-53 / 1e-6 of the loss's terms stay below)."""
    print(f"[case] slopes {shape}", flush=True)
    cfg, p, d, b, spans, dy, q, ref, tol = inputs(moe, shape, 61)
    dx, dw = backward(moe, p, d, b, dy)
    torch.cuda.synchronize()
    got = {"x": dx, **dw}
    t = 1e-6
    for n in NAMES:
        v = torch.sign(ref[n])
        slope = float((forward({**q, n: q[n] + t * v}, spans, dy)
                       - forward({**q, n: q[n] - t * v}, spans, dy)) / (2 * t))
        # the 64-bit gradient, without the kernels' roundings
        assert abs(float((ref[n] * v).sum()) - slope) <= 1e-5 * abs(slope), n
        allowed = float(tol[n].sum()) + 1e-5 * abs(slope)
        along = float((got[n].double() * v).sum())
        assert abs(along - slope) <= allowed, n
        for wrong in (0.0, -along, 0.5 * along):
            assert abs(wrong - slope) > allowed, (n, "a wrong gradient passes")
