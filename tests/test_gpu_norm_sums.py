"""The norm's sums and its gradient's, held to the additions that the kernels
make one after the other (U = 2^-24, half a step of fp32):

 - over a row: at most 16 values in a lane, 6 steps over a wave, up to 16 waves:
   38 additions;
 - over rows: a group of lanes adds every (number of groups)-th row, up to 4
   groups of a workgroup are added, then every 16th of the workgroups' sums, then
   16 of those.  A workgroup leaves 8 H bytes in the workspace, which tells how
   many there are.

The mean of a row is off by m = 39 U mean|x| (the sum and the division); a
deviation d = x - mean by U |d| and m; their squares' mean, 3 U from the squares
and 38 from the sum and 2 from the division and eps, by 43 U of itself and by m^2
(the deviations add up to 0); r by half of that, the root and the quotient.
In the gradient mean and r are given: xh = (x - mean) r is off by 2 U, g = dy w
by U, g xh by 4 U, its mean by 44 U, that of g by 41 U.  One percent is added for
the products of errors."""
import pytest
import torch

from test_gpu_norm import BF16, F32, U, backward64, forward64, half_step, inputs

pytestmark = pytest.mark.gpu

SIZES = [(1, 8), (700, 64), (5000, 512), (3000, 520), (3000, 1000), (2500, 2048), (2000, 4096), (1500, 5120), (1100, 8192),
         (600, 8200), (9, 16384), (700, 16384)]


@pytest.fixture(scope="module")
def moe():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    from group_limited_routing_router_amd import moe as m
    m.load_library()
    return m


def worst(got, ref, tol):
    return float(((got.double() - ref).abs() / (1.01 * tol + 1e-30)).max())


@pytest.mark.parametrize("center", [False, True], ids=["rms", "layer"])
@pytest.mark.parametrize("x_dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("rows,H", SIZES)
def test_forward(moe, rows, H, x_dtype, center):
    print(f"[case] norm sums {rows} {H} {x_dtype} {center}", flush=True)
    x, w, b, _ = inputs(rows, H, x_dtype, F32, rows + H, center)
    out, stats = torch.full((rows, H), float("nan"), device="cuda"), torch.full((rows, 2), float("nan"), device="cuda")
    moe.moe_norm(x, w, b, 1e-6, out, stats, center=center)
    x64, w64, b64 = x.double(), w.double(), b.double()
    ref, mean, r = forward64(x64, w64, b64, 1e-6, center)
    m = 39 * U * x64.abs().mean(dim=1, keepdim=True) if center else torch.zeros_like(mean)
    dr = r * (21.5 * U + (m * r).square() / 2 + 2 * U)
    d = (x64 - mean).abs()
    tol = w64.abs() * (d * dr + m * r + 3 * U * d * r) + U * (ref.abs() + b64.abs())
    assert worst(stats[:, :1], mean, m + U * mean.abs()) <= 1.0
    assert worst(stats[:, 1:], r, dr) <= 1.0
    assert worst(out, ref, tol) <= 1.0
    half = torch.empty((rows, H), dtype=BF16, device="cuda")
    moe.moe_norm(x, w, b, 1e-6, half, center=center)
    assert torch.equal(half, out.to(BF16))  # rounded once


@pytest.mark.parametrize("center", [False, True], ids=["rms", "layer"])
@pytest.mark.parametrize("types", [(F32, BF16), (BF16, BF16)], ids=["f32", "bf16"])
@pytest.mark.parametrize("rows,H", SIZES)
def test_backward(moe, rows, H, types, center):
    print(f"[case] norm gradient sums {rows} {H} {types} {center}", flush=True)
    x, w, b, dy = inputs(rows, H, *types, rows * 3 + H, center)
    _, mean, r = forward64(x.double(), w.double(), None, 1e-6, center)
    stats = torch.cat([mean, r], dim=1).float().contiguous()
    mean, r = stats[:, :1].double(), stats[:, 1:].double()
    x64, w64, dy64 = x.double(), w.double(), dy.double()
    ref, rw, rb = backward64(dy64, x64, w64, mean, r, center)
    xh, g = ((x64 - mean) * r).abs(), (dy64 * w64).abs()
    along, level = (g * xh).mean(dim=1, keepdim=True), g.mean(dim=1, keepdim=True)
    if not center:
        level = torch.zeros_like(level)
    tol = r * U * (g + 3 * xh * along + 44 * xh * along + 41 * level + 2 * (g + xh * along + level)) + U * ref.abs()
    bytes_ = moe.moe_norm_workspace_bytes(rows, H)
    parts = bytes_ // (8 * H)
    groups = 4 if H <= 512 else 1  # of a workgroup
    steps = -(-rows // (parts * groups)) + groups + -(-parts // 16) + 16
    tw, tb = (3 + steps) * U * (dy64.abs() * xh).sum(dim=0), steps * U * dy64.abs().sum(dim=0)
    ws = torch.full((bytes_,), 0xFF, dtype=torch.uint8, device="cuda")
    dx = torch.full((rows, H), float("nan"), device="cuda")
    dw, db = torch.full((H,), float("nan"), device="cuda"), torch.full((H,), float("nan"), device="cuda")
    moe.moe_norm_backward(dy, x, w, stats, dx, dw, db, ws, center=center)
    assert worst(dx, ref, tol) <= 1.0
    assert worst(dw, rw, tw) <= 1.0 and worst(db, rb, tb) <= 1.0
    half = torch.empty((rows, H), dtype=BF16, device="cuda")
    moe.moe_norm_backward(dy, x, w, stats, half, dw, db, ws, center=center)
    assert torch.equal(half, dx.to(BF16)) and half_step(BF16) == 2.0 ** -8
