"""The FP8 experts on operands whose sums are exact, and what the kernels may
then be off by.

x and dy are whole numbers up to 8 (times a power of two), which are e4m3 codes
exactly; weights are codes of whole numbers up to 8 with scales of one power of
two and its neighbours.  Products of two codes are whole numbers of at most 11
bits, which the matrix instructions do not cut, and their sums stay below 2^24
units, so g, u and dh are exact in fp32.  What is left:

 - the activation in fp32 (u = 2^-24, half a step): s = 1 / (1 + exp(-g)) is off
   by 6 u s (exp 4, of which exp(-g) / (1 + exp(-g)) <= 1 counts, the sum 1, the
   division 1), silu = g s by 7 u, 1 - s by 6 u s + u (1 - s).  With S = |silu|
   the slope s + silu (1 - s) is off by u (6 s + 9 S (1 - s) + 6 S s) and the last
   sum's u (s + S (1 - s)); the two products beside it 2 u of the result.  One
   percent is added for the products of these.
 - the roundings to e4m3 codes and to bf16 are those of the definition.  Only
   where a value lies so close to a border that the above decides may the kernel
   take the other side: the spread of the value's roundings over its range.
 - dx is a sum of code products that are not whole: 7 x 2^-13 of the sum of
   magnitudes and (length / 8 + 32) 2^-23 of it, as counted in _fp8block.py; the
   weights' gradients are sums of exact products of bf16 in fp32, rows / 16 + 32
   steps of 2^-23, as counted in _grouped.py."""
import torch

import _fp8block as f8
from _grouped import counts_for, offsets_of
from group_limited_routing_router_amd.moe import MoEProblem

import numpy as np

NAMES = ("gate", "up", "down")
U = 2.0 ** -24
BF16, F32 = torch.bfloat16, torch.float32


def on(device, t):
    return t.to(device) if t is not None else None


class WholeExperts:
    """Tokens, weights and gradients of one shape on `device`."""

    def __init__(self, T, k, E, H, I, seed=0, kind="random", counts=None, device="cpu", order=False):
        rng = np.random.default_rng(seed)
        gen = torch.Generator(device=device).manual_seed(seed)
        self.T, self.k, self.E, self.H, self.I, self.P, self.device = T, k, E, H, I, T * k, device
        self.counts = counts_for(self.P, E, kind, rng) if counts is None else counts
        assert int(self.counts.sum()) == self.P
        self.offsets = offsets_of(self.counts).to(device)
        pairs = np.arange(self.P) if order else rng.permutation(self.P)
        self.pairs = torch.from_numpy(pairs.astype(np.int32)).to(device)
        self.rows = self.pairs.long() // k

        def whole(*shape):
            return torch.randint(-8, 9, shape, generator=gen, device=device)

        self.x = whole(T, H).to(BF16)
        self.dy = (whole(self.P, H) * 2.0 ** -6).to(BF16)
        table = f8.code_of(torch.arange(-8, 9).double()).to(device)
        self.q, self.s = {}, {}
        # gates of a few units: whole numbers up to 8 are 4.9 in the mean square
        for name, N, K in (("gate", I, H), ("up", I, H), ("down", H, I)):
            self.q[name] = table[whole(E, N, K) + 8]
            unit = 127 - round(float(np.log2(12.0 * np.sqrt(H))))
            self.s[name] = torch.randint(unit - 1, unit + 2, (E, f8.blocks(N), f8.blocks(K)), generator=gen,
                                         device=device, dtype=torch.uint8)
            # every sum of magnitudes in units of the smallest scale
            assert 64 * 4 * K < 2 ** 24

    def problem(self):
        return MoEProblem(self.T, self.H, self.I, self.E, 1, 1, self.k, 1.0)

    def weights(self):
        return [t[n] for n in NAMES for t in (self.q, self.s)]

    def spans(self):
        o = self.offsets.tolist()
        return [(e, o[e], o[e + 1]) for e in range(self.E) if o[e + 1] > o[e]]

    def matrix(self, name, e):
        return f8.value_weights(self.q[name][e:e + 1], self.s[name][e:e + 1])[0]


def blockwise(v, off, edge):
    """The rows of v in 64 bits, off by up to `off`, rounded to codes by blocks
    of 128: the value of the definition and how far another rounding inside that
    range may lie from it."""
    n = v.shape[1]
    pad = lambda t: torch.nn.functional.pad(t, (0, -n % 128)).reshape(len(t), -1, 128)  # noqa: E731
    p, o = pad(v), pad(off)

    def rounded(x, top):
        e, _, tiny = f8.scale_exponents(top)
        assert not tiny[top > 0].any()
        s = torch.exp2(e)[:, :, None]
        return (f8.to_e4m3(x / s) * s).reshape(len(v), -1)[:, :n]

    top = p.abs().amax(2)
    mid = rounded(p, top)
    spread = torch.zeros_like(mid)
    for t in ((p.abs() - o).clamp(min=0).amax(2), (p.abs() + o).amax(2)):
        for x in (p - o, p + o):
            spread = torch.maximum(spread, (rounded(x, t) - mid).abs())
    edge.append((int((spread > 0).sum()), spread.numel()))
    return mid, spread


def halved(v, off, edge):
    """As blockwise, to bf16."""
    r = lambda x: x.float().to(BF16).double()  # noqa: E731  (64 to 32 bits first: counted in off)
    mid = r(v)
    spread = torch.maximum((r(v - off) - mid).abs(), (r(v + off) - mid).abs())
    edge.append((int((spread > 0).sum()), spread.numel()))
    return mid, spread


def gradients(c):
    """(reference, tolerance) in 64 bits of dx, dw_gate, dw_up and dw_down with
    fp32 outputs; asserts that next to no rounding is open."""
    x, dy = c.x.double()[c.rows], c.dy.double()
    new = lambda *s: torch.zeros(s, dtype=torch.float64, device=c.device)  # noqa: E731
    dx, tx = new(c.P, c.H), new(c.P, c.H)
    dw = {n: new(*c.q[n].shape) for n in NAMES}
    tw = {n: new(*c.q[n].shape) for n in NAMES}
    edge = []
    for e, i, j in c.spans():
        wg, wu, wd = (c.matrix(n, e) for n in NAMES)
        g, u, dh = x[i:j] @ wg.T, x[i:j] @ wu.T, dy[i:j] @ wd
        s = 1 / (1 + torch.exp(-g))
        silu = g * s
        S = silu.abs()
        dg, du, h = dh * u * (s + silu * (1 - s)), dh * silu, silu * u
        # the definition's own rounding to 32 bits is one more U of the value
        og = 1.01 * U * (dh * u).abs() * (9 * s + 12 * S * (1 - s) + 6 * S * s) + U * dg.abs()
        ou, oh = 1.01 * U * 9 * du.abs(), 1.01 * U * 9 * h.abs()
        cuts = f8.CUT + (c.I / 4 + 32) * 2.0 ** -23
        for v, off, w in ((dg, og, wg), (du, ou, wu)):
            mid, spread = blockwise(v, off, edge)
            dx[i:j] += mid @ w
            open_ = spread @ w.abs()
            tx[i:j] += open_ + cuts * (mid.abs() @ w.abs() + open_)
        sums = ((j - i) / 16 + 32) * 2.0 ** -23
        gb, gs = halved(dg, og, edge)
        ub, us = halved(du, ou, edge)
        hb, hs = halved(h, oh, edge)
        for n, l, ls, r, rs in (("gate", gb, gs, x[i:j], None), ("up", ub, us, x[i:j], None),
                                ("down", dy[i:j], None, hb, hs)):
            dw[n][e] = l.T @ r
            open_ = ls.T @ r.abs() if rs is None else l.abs().T @ rs
            tw[n][e] = open_ + sums * (l.abs().T @ r.abs() + open_)
    # a rounding is open where a value lies within a few U of a border: codes
    # have borders every 2^-4 of a value or so, bf16 every 2^-8
    assert sum(a for a, _ in edge) <= 0.01 * sum(b for _, b in edge) + 2
    return [(dx, tx)] + [(dw[n], tw[n]) for n in NAMES]


def off_by(got, ref, tol, dtype):
    """The largest error in tolerances; a bf16 output adds half a step."""
    t = tol + torch.finfo(dtype).eps / 2 * (ref.abs() + tol) + 1e-30
    v = (got.double() - ref).abs() / t
    return float(torch.nan_to_num(v, nan=float("inf")).max()) if v.numel() else 0.0
