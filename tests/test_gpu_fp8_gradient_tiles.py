"""The FP8 experts and their gradients on 128- and 256-row tiles, for every number
of rows of an expert: every count of row blocks of a wave, and blocks that end at
every row."""
import numpy as np
import pytest
import torch

import test_gpu_fp8_limits as limits
from _grouped import offsets_of
from test_gpu_fp8_experts import NAMES, Experts, backward, reference_gradients, within

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def moe():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    from group_limited_routing_router_amd import moe as m
    m.load_library()
    return m


def test_every_count_of_rows(moe):
    counts = np.random.default_rng(3).permutation(np.arange(1, 257))
    c = Experts(int(counts.sum()), 1, 256, 128, 192, seed=3)
    c.counts, c.offsets = counts, offsets_of(counts)
    dx, dw = backward(moe, c)
    torch.cuda.synchronize()
    rdx, tx, rdw, tw = reference_gradients(c)
    worst = [within(dx[i:j], rdx[i:j], tx[i:j], F32) for _, i, j in c.spans()]
    assert max(worst) <= 1.0, [int(counts[e]) for e, w in enumerate(worst) if w > 1.0]
    for n in NAMES:
        worst = [within(dw[n][e], rdw[n][e], tw[n][e], F32) for e in range(256)]
        assert max(worst) <= 1.0, (n, [int(counts[e]) for e, w in enumerate(worst) if w > 1.0])


@pytest.mark.parametrize("left", [1, 32, 33, 64, 70, 96, 97, 127, 128, 129, 160, 161, 192, 200, 224, 225, 255])
def test_dense_rows(moe, left):
    """A dense layer without a dispatch is the one with the dispatch written out,
    to the bit; the last tile has `left` rows."""
    c = Experts(256 * 64 + left, 1, 1, 128, 512, seed=4)
    c.pairs = torch.arange(c.P, dtype=torch.int32)
    c.rows = c.pairs.long()
    want = backward(moe, c)
    c.dispatch = lambda: (None, None)
    got = backward(moe, c)
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.isfinite(want[0]).all()
    for n in NAMES:
        assert torch.equal(got[1][n], want[1][n])


def every_count(monkeypatch, most):
    counts = np.random.default_rng(most).permutation(np.arange(1, most + 1))
    monkeypatch.setattr(limits, "draw_counts", lambda gen, P, E: counts)
    return int(counts.sum())


@pytest.mark.parametrize("op", ["product", "input_grad"])
@pytest.mark.parametrize("most,N,K", [(256, 1040, 1024), (128, 272, 256)])
def test_products(moe, monkeypatch, op, most, N, K):
    limits.test_tiles(moe, op, (every_count(monkeypatch, most), most, N, K))


@pytest.mark.parametrize("most", [256, 128])
def test_gated(moe, monkeypatch, most):
    limits.test_gated_tiles(moe, every_count(monkeypatch, most), most, 256, 192)


def test_every_count_of_rows_small(moe):
    """As above on 128 rows."""
    counts = np.random.default_rng(5).permutation(np.arange(1, 129))
    c = Experts(int(counts.sum()), 1, 128, 128, 192, seed=5)
    c.counts, c.offsets = counts, offsets_of(counts)
    dx, dw = backward(moe, c)
    torch.cuda.synchronize()
    rdx, tx, rdw, tw = reference_gradients(c)
    assert within(dx, rdx, tx, F32) <= 1.0
    for n in NAMES:
        assert within(dw[n], rdw[n], tw[n], F32) <= 1.0
