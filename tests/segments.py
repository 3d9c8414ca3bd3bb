"""Packed expert rows for the tests of the experts' training and 8-bit calls:
inputs over given segment lengths, and their gated blocks in 64 bits.

Rows behind the last segment hold NaN in every input (a call that read them
would spread it) and a sentinel in every output (a call that wrote them would
lose it).
"""
import numpy as np
import torch

import combine_router_top_amd as M

SENTINEL = -77.0
# half a step of each type, relative to the value
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}


def torch_dtype(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def spec(counts, d, f, dtype, T=None, k=None, E=None):
    """A problem whose buffers hold sum(counts) rows and T >= max(counts)."""
    n = len(counts)
    T = max(1, max(counts)) if T is None else T
    k = min(n, -(-max(1, sum(counts)) // T)) if k is None else k
    p = M.Spec(T, d, n if E is None else E, k, f, 0, n, dtype)
    assert p.rows_max >= sum(counts) and p.k <= 32
    return p


def offsets_of(counts):
    return torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32).cuda()


class Rows:
    """Seeded inputs: float64 values that the storage type holds exactly."""

    def __init__(self, p, counts, seed):
        self.p, self.counts, self.A = p, list(counts), int(sum(counts))
        self.bounds = np.concatenate([[0], np.cumsum(counts)]).astype(int)
        self.gen = torch.Generator().manual_seed(seed)
        self.dt = torch_dtype(p.dtype)

    def draw(self, *shape, scale=1.0):
        return (torch.randn(shape, generator=self.gen) * scale).to(self.dt).double()

    def dev(self, v):
        return v.to(self.dt).cuda()

    def packed(self, v):
        """[A, w] values on the device in a buffer of rows_max rows, NaN behind."""
        t = torch.full((self.p.rows_max, v.shape[1]), float("nan"), dtype=self.dt)
        t[: self.A] = v.to(self.dt)
        return t.cuda()

    def out(self, width):
        return torch.full((self.p.rows_max, width), SENTINEL, dtype=self.dt, device="cuda")

    def check_tail(self, *outs):
        for o in outs:
            assert bool((o[self.A:] == SENTINEL).all()), "rows behind the last segment were written"

    def segments(self):
        return [(e, slice(int(self.bounds[e]), int(self.bounds[e + 1]))) for e in range(len(self.counts))]


def assert_within(got, ref, tol, what):
    """|got - ref| <= tol elementwise (float64 tensors; tol derived by the caller)."""
    got = got.detach().cpu().double()
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    assert bool(torch.isfinite(got).all()), f"{what}: non-finite values"
    over = ((got - ref).abs() - tol)
    if over.numel():
        worst = over.max().item()
        at = np.unravel_index(int(over.argmax()), over.shape)
        assert worst <= 0, f"{what}: {got[at]:.6g} against {ref[at]:.6g}, allowed {tol[at]:.3g} at {at}"


def dot_slack(a, b):
    """Bound of the fp32 error of the product a b: every one of the K additions
    rounds a partial sum of at most sum |a b| (2^-23: also where it truncates)."""
    return a.shape[1] * 2.0 ** -23 * (a.abs() @ b.abs())
