"""Sampling over rows with many equal logits of small weights, where a rounding of one weight counts as often as there are
copies of it.

A decision (where a filter cuts, which token the given number falls on) may differ from that of the definition only where the
definition's own comparison is within 1e-12 of the sum.  That bound: a weight is right to 2^-41.5 of itself (the exponential's
pairs of fp32 numbers) and rounded to a unit that is 2^-60 of the row's sum at most, and what is below 2^-60 of the largest weighs
nothing; with V = 393,216 of them 3.2e-13 + V (2^-61 + 2^-60) < 0.9e-12.  Here both sides of each comparison are computed as
rational numbers from exp() in double precision, whose own 2^-52 is far below that."""
from fractions import Fraction
import math

import numpy as np
import pytest

import bit_affine_quantized_mlx_gb300 as q4

pytestmark = pytest.mark.gpu
NEAR = Fraction(1, 10 ** 12)


@pytest.fixture(scope="module")
def torch():
    import torch
    import __graft_entry__
    __graft_entry__.build()
    return torch


class Row:
    """One row of few distinct logits: the order (logit descending, index ascending) as runs of equals."""

    def __init__(self, logits, t):
        self.logits = logits
        values, inverse, counts = np.unique(-logits, return_inverse=True, return_counts=True)
        self.place = inverse  # run of each token
        self.counts = [int(c) for c in counts]
        self.w = [Fraction(math.exp(-(v - values[0]) / t)) for v in values.tolist()]
        # how many of a token's equals come before it
        order = np.argsort(inverse, kind="stable")
        self.nth = np.empty(len(logits), np.int64)
        start = np.concatenate([[0], np.cumsum(counts)])
        self.nth[order] = np.arange(len(logits)) - start[inverse[order]]

    def sum_of(self, n):
        """Of the first n tokens of the order."""
        total = Fraction(0)
        for c, w in zip(self.counts, self.w):
            total += min(n, c) * w
            n -= min(n, c)
        return total

    def kept_by(self, n):
        """A token is kept if fewer than keep[run] of its equals come before it."""
        keep = []
        for c in self.counts:
            keep.append(min(n, c))
            n -= keep[-1]
        return np.array(keep)

    def before(self, token, keep):
        """Sum of the kept tokens of lower index."""
        total = Fraction(0)
        runs = self.place[:token]
        kept = runs[self.nth[:token] < keep[runs]]
        for run, count in zip(*np.unique(kept, return_counts=True)):
            total += int(count) * self.w[run]
        return total


def check(torch, logits, dtype, us, t=1.0, k=None, p=None, m=None):
    """One row of logits (float64 values that dtype holds), drawn from once for each of us."""
    row = Row(logits, t)
    B, V = len(us), len(logits)
    l = torch.from_numpy(logits).to(getattr(torch, dtype)).cuda()
    assert bool((l.double().cpu() == torch.from_numpy(logits)).all())
    full = lambda v, kind: None if v is None else torch.full((B,), v, dtype=kind, device="cuda")
    op = q4.Sampling(full(t, torch.float32), full(k, torch.int32), full(p, torch.float32), full(m, torch.float32))
    u = torch.tensor(np.asarray(us, np.float32)).cuda()
    token, kept = (torch.full((B,), -7, dtype=torch.int32, device="cuda") for _ in "tk")
    ws = q4.new_workspace(q4.lily_sample_workspace_bytes(B, V))
    q4.lily_sample(op, l[None].expand(B, V), u, token, kept=kept, ws=ws)
    assert q4.lily_q4_workspace_status(ws) == q4.OK
    assert len(set(kept.tolist())) == 1
    n = int(kept[0])
    assert 1 <= n <= V
    most = min(k, V) if k else V
    whole = row.sum_of(most)
    if p is not None and p < 1:
        target = Fraction(float(np.float32(p))) * whole
        assert n <= most
        assert row.sum_of(n) >= target - NEAR * whole, ("too few", n)
        assert n == 1 or row.sum_of(n - 1) < target + NEAR * whole, ("too many", n)
    elif m:
        assert n == min(most, sum(c for c, w in zip(row.counts, row.w) if w >= Fraction(float(np.float32(m)))))
    else:
        assert n == most
    keep, total = row.kept_by(n), row.sum_of(n)
    for value, at in zip(u.tolist(), token.tolist()):
        run = row.place[at]
        assert row.nth[at] < keep[run], ("not kept", at)
        place, from_ = Fraction(min(value, 1 - 2.0 ** -24)) * total, row.before(at, keep)  # 1 and beyond: as at the end
        assert from_ - NEAR * total <= place < from_ + row.w[run] + NEAR * total, (value, at, float((place - from_) / row.w[run]))


def flat(V, tail, peak_at=0, peak=0.0):
    l = np.full(V, tail)
    l[peak_at] = peak
    return l


def spread(n, lo, hi, seed=0):
    return np.random.default_rng(seed).uniform(lo, hi, n).astype(np.float32)


@pytest.mark.parametrize("dtype,V,tail,p", [("bfloat16", 151936, -27.25, 1 - 2.0 ** -24), ("float16", 151936, -25.109375, 0.999999),
                                            ("float16", 151936, -18.234375, 0.999), ("float32", 393216, -26.3, 0.9999999),
                                            ("float32", 50257, -20.1, 0.99999), ("float16", 393216, -12.0078125, 0.5),
                                            ("float32", 3001, -23.7, 0.99999997)])
@pytest.mark.parametrize("last", [False, True])
def test_cut_in_a_flat_tail(torch, dtype, V, tail, p, last):
    tail = float(np.float32(tail))
    check(torch, flat(V, tail, V - 1 if last else 0), dtype, [0.0, 0.3, 0.99999], p=p)


@pytest.mark.parametrize("V", [6000, 151936])
def test_cut_in_steps(torch, V):
    """Some dozens of distinct logits with thousands of copies each, as rows of 16 bits have them."""
    rng = np.random.default_rng(V)
    l = np.round(rng.normal(-14, 2.2, V) * 16) / 16
    l[rng.choice(V, 20, replace=False)] = np.round(rng.normal(7, 3, 20) * 16) / 16
    for t, p in ((0.8, 0.99999), (1.0, 1 - 2.0 ** -24), (1.3, 0.9999), (1.0, 0.9999999)):
        check(torch, l, "float16", [0.1, 0.9999999], t=float(np.float32(t)), p=p)


@pytest.mark.parametrize("V,tail", [(151936, -27.25), (393216, -22.875), (393216, -29.5)])
def test_the_token_in_a_flat_tail_after_a_cut(torch, V, tail):
    w = math.exp(tail)
    us = np.concatenate([spread(20, 0, V * w / (1 + V * w)), [0.0, 0.5]])
    for kw in (dict(p=1 - 2.0 ** -24), dict(k=V - 5), dict(m=1e-14), dict(k=V - 3, p=0.99999994), dict(k=400)):
        check(torch, flat(V, tail, V - 1), "bfloat16", us, **kw)


def test_short_lists(torch):
    """What a list holds weighs as much as sums over the row do."""
    for n, peak in ((2, 3), (100, 3), (500, 3), (2, 19999), (100, 19999), (500, 19999)):
        l = np.full(20000, -300.0)
        l[7:7 + 39 * n:39] = -24.5
        l[peak] = 0.0
        w = math.exp(-24.5)
        us = np.concatenate([[0.0, 0.5], 1 - spread(10, 0, n * w), spread(10, 0, n * w)])
        for kw in (dict(p=0.99999994), dict(k=300), dict(k=n, p=0.99999994), dict(m=1e-12)):
            check(torch, l, "bfloat16", us, **kw)


@pytest.mark.parametrize("V,tail", [(151936, -27.25), (393216, -29.5), (393216, -36.25)])
def test_the_token_in_a_flat_tail(torch, V, tail):
    """Without a filter, where weights are too small for the sums that are not exact to decide."""
    w = math.exp(tail)
    check(torch, flat(V, tail, V - 1), "bfloat16", np.concatenate([spread(30, 0, V * w / (1 + V * w)), [0.0, 0.5]]))
