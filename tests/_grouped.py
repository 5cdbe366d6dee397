"""Inputs and 64-bit references of the grouped products, and their tolerances.

fp32 outputs: the products of two bf16 values are exact in fp32; the matrix
instructions add 16 of them to an accumulator at a time, so a sum of R
products takes R / 16 steps and each step's additions are off by at most
2^-23 of the sum of magnitudes S (twice the half step of fp32, for an adder
that drops bits); the 16 additions inside a step and the joins of a split sum
count 32 more.  |error| <= (R / 16 + 32) 2^-23 S.  A bf16 output adds half a
step of its own, 2^-8 of the value (and of the error before it)."""
import numpy as np
import torch

from group_limited_routing_router_amd.moe import MoEGemmProblem


def offsets_of(counts, first=0):
    off = np.zeros(len(counts) + 1, np.int32)
    off[0] = first
    off[1:] = first + np.cumsum(counts)
    return torch.from_numpy(off)


def counts_for(P, E, kind, rng):
    """Rows of each expert, P in all: even, random (some idle), or all but a
    few on one expert."""
    if kind == "even":
        return np.array([P // E + (e < P % E) for e in range(E)])
    if kind == "one":
        c = np.zeros(E, np.int64)
        c[rng.integers(E)] = P
        return c
    p = rng.exponential(1.0, E) * (rng.random(E) > 0.3) + 1e-9
    return rng.multinomial(P, p / p.sum())


def problem(P, S, E, N, K, k=1):
    return MoEGemmProblem(P, S, E, N, K, k)


class Case:
    """Inputs of every grouped product of one shape: P positions of which the
    first `first` and the last `behind` belong to no expert.  The references
    are computed on `device`."""

    def __init__(self, P, E, N, K, k=1, kind="random", seed=0, first=0, behind=0, S=None,
                 device="cpu"):
        rng = np.random.default_rng(seed)
        gen = torch.Generator().manual_seed(seed)
        self.P, self.E, self.N, self.K, self.k = P, E, N, K, k
        self.counts = counts_for(P - first - behind, E, kind, rng)
        self.offsets = offsets_of(self.counts, first)
        if k > 1:
            self.S = -(-P // k) if S is None else S
            pairs = rng.permutation(self.S * k)[:P].astype(np.int32)
            self.pairs = torch.from_numpy(pairs)
            self.rows = self.pairs.long() // k
        else:
            self.S, self.pairs, self.rows = P if S is None else S, None, torch.arange(P)
        self.a = torch.randn((self.S, K), generator=gen).to(torch.bfloat16)
        self.w = (0.05 * torch.randn((E, N, K), generator=gen)).to(torch.bfloat16)
        self.dout = (0.1 * torch.randn((P, N), generator=gen)).to(torch.bfloat16)
        self.a8 = torch.randint(-128, 128, (self.S, K), generator=gen, dtype=torch.int8)
        self.w8 = torch.randint(-128, 128, (E, N, K), generator=gen, dtype=torch.int8)
        self.a_scale = torch.rand((self.S,), generator=gen) * 0.05 + 1e-3
        self.w_scale = torch.rand((E, N), generator=gen) * 0.01 + 1e-4
        for name in ("a", "w", "dout", "a8", "w8", "a_scale", "w_scale", "rows"):
            setattr(self, name, getattr(self, name).to(device))

    def problem(self):
        return problem(self.P, self.S, self.E, self.N, self.K, self.k)

    def spans(self):
        off = self.offsets.tolist()
        return [(e, off[e], off[e + 1]) for e in range(self.E) if off[e + 1] > off[e]]

    def owned(self):
        m = torch.zeros(self.P, dtype=torch.bool)
        m[int(self.offsets[0]):int(self.offsets[-1])] = True
        return m

    # each reference: (value, sum of magnitudes, length of the sum) in 64 bits
    def product(self):
        v = torch.zeros((self.P, self.N), dtype=torch.float64, device=self.a.device)
        m = torch.zeros_like(v)
        for e, i, j in self.spans():
            a, w = self.a[self.rows[i:j]].double(), self.w[e].double()
            v[i:j] = a @ w.T
            m[i:j] = a.abs() @ w.abs().T
        return v, m, self.K

    def input_grad(self):
        v = torch.zeros((self.P, self.K), dtype=torch.float64, device=self.a.device)
        m = torch.zeros_like(v)
        for e, i, j in self.spans():
            d, w = self.dout[i:j].double(), self.w[e].double()
            v[i:j] = d @ w
            m[i:j] = d.abs() @ w.abs()
        return v, m, self.N

    def weight_grad(self):
        v = torch.zeros((self.E, self.N, self.K), dtype=torch.float64, device=self.a.device)
        m = torch.zeros_like(v)
        for e, i, j in self.spans():
            d, a = self.dout[i:j].double(), self.a[self.rows[i:j]].double()
            v[e] = d.T @ a
            m[e] = d.abs().T @ a.abs()
        return v, m, int(self.counts.max()) if self.E else 0

    def int8(self):
        """The int8 product exactly as defined: an exact sum, rounded to fp32,
        times the fp32 product of the scales."""
        v = torch.zeros((self.P, self.N), dtype=torch.float32, device=self.a.device)
        for e, i, j in self.spans():
            acc = self.a8[self.rows[i:j]].double() @ self.w8[e].double().T
            v[i:j] = acc.float() * (self.a_scale[self.rows[i:j]][:, None] * self.w_scale[e][None, :])
        return v


def tolerance(ref, magnitudes, length, dtype, start=None):
    """The largest |error| of each element; start: what accumulate adds to
    (one more fp32 addition)."""
    t = (length / 16 + 32) * 2.0 ** -23 * magnitudes
    if start is not None:
        t = t + 2.0 ** -24 * (start.double().abs() + ref.abs())
    if dtype == torch.bfloat16:
        t = t + 2.0 ** -8 * (ref.abs() + t)
    return t + 1e-30


def worst(got, ref, tol):
    """max |got - ref| / tolerance; NaN in got counts as infinite."""
    if ref.numel() == 0:
        return 0.0
    x = ((got.double() - ref).abs() / tol)
    return float(torch.nan_to_num(x, nan=float("inf")).max())
