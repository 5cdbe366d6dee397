"""The check of the FP8 experts' gradients (_fp8exact.py) fails for wrong ones,
and the shapes of the GPU tests reach every tile of the two-matrix product and
of the gated pass."""
import pytest
import torch

from _fp8exact import F32, NAMES, WholeExperts, blockwise, gradients, off_by
from _fp8plan import plan
from test_gpu_fp8_exact import DENSE, SHAPES, tiles_of

SMALL = [(300, 1, 2, 640, 704), (9, 1, 1, 2560, 384), (64, 8, 16, 256, 448), (40, 2, 3, 128, 320)]


@pytest.mark.parametrize("shape", SMALL, ids=str)
def test_wrong_gradients_are_rejected(shape):
    c = WholeExperts(*shape, seed=1)
    right = gradients(c)
    for ref, tol in right:
        assert off_by(ref.float(), ref, tol, F32) <= 1.0
        for wrong in (ref * 0.5, ref * 0, -ref, ref * 1.1):
            assert off_by(wrong, ref, tol, F32) > 1.0
        # nearly every element by itself shows a half of it
        shown = (0.5 * ref.abs() > tol)[ref != 0].double().mean()
        assert shown > 0.9, shown
    (dx, tx), *_ = right
    # one block of 128 of dg left out of the reduction, or its scale off by two
    e, i, j = max(c.spans(), key=lambda t: t[2] - t[1])
    x, dy = c.x.double()[c.rows][i:j], c.dy.double()[i:j]
    wg, wu, wd = (c.matrix(n, e) for n in NAMES)
    g, u, dh = x @ wg.T, x @ wu.T, dy @ wd
    s = 1 / (1 + torch.exp(-g))
    mid, _ = blockwise(dh * u * s * (1 + g * (1 - s)), torch.zeros_like(g), [])
    for b in range(0, c.I, 128):
        part = mid[:, b:b + 128] @ wg[b:b + 128]
        for wrong in (dx[i:j] - part, dx[i:j] + part, dx[i:j] - 0.5 * part):
            assert off_by(wrong, dx[i:j], tx[i:j], F32) > 1.0
    # one row of the largest expert taken from its neighbour
    if j - i > 1:
        wrong = dx.clone()
        wrong[i] = dx[i + 1]
        assert off_by(wrong, dx, tx, F32) > 1.0


def test_formulas_against_automatic_differentiation():
    """The references without their roundings."""
    c = WholeExperts(12, 2, 3, 128, 64, seed=2)
    x = c.x.double()[c.rows].requires_grad_()
    w = [torch.stack([c.matrix(n, e) for e in range(c.E)]).requires_grad_() for n in NAMES]
    total = 0.0
    for e, i, j in c.spans():
        g, u = x[i:j] @ w[0][e].T, x[i:j] @ w[1][e].T
        total = total + (c.dy.double()[i:j] * ((g / (1 + torch.exp(-g)) * u) @ w[2][e].T)).sum()
    want = torch.autograd.grad(total, [x, *w])
    # roundings of 2^-4 of the terms of dx, 2^-8 of the weights' gradients, either way
    for (ref, _), true, near in zip(gradients(c), want, (0.1, 0.01, 0.01, 0.01)):
        assert float((ref - true).norm() / true.norm()) < near


def test_shapes_reach_every_tile():
    pairs, gated = set(), set()
    for (T, k, E, H, I), want in SHAPES.items():
        assert tiles_of(T, k, E, H, I) == want, (T, k, E, H, I)
        (rows, nt, splits), (grows, gnt, _) = want
        stages = 2 * -(-I // 128)
        pairs.add((rows, nt, splits > 1, stages // splits > 40))
        gated.add((grows, gnt))
    assert gated == {(32, False), (32, True), (128, False), (128, True), (256, False)}
    assert {(r, n) for r, n, _, _ in pairs} == {(32, False), (32, True), (128, False), (128, True), (256, False)}
    # split and not, more stages than scales held in registers and fewer
    for rows in (32, 128, 256):
        assert {s for r, _, s, _ in pairs if r == rows} == {False, True}
        assert {x for r, _, _, x in pairs if r == rows} == {False, True}


def test_dense_shapes_reach_every_ungathered_tile():
    got = {plan("gated", T, 1, I, H)[:2] for T, H, I in DENSE}
    assert got == {(32, False), (32, True), (128, False), (128, True), (256, False)}
