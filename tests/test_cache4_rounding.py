"""Attention over the 4-bit cache where few keys carry the weight: its outputs are
as near to the definition as one rounding to bf16 leaves them.

Let x be what a kernel sums in fp32, w the definition's value and r(v) = |bf16(v) - v|.
r moves by no more than its argument, so |bf16(x) - w| <= r(w) + 2 |x - w|, and the norms over
all outputs keep |got - w| <= |r(w)| + 2 |x - w|.  x - w is, of what the sums add up,

    2^-16     P s in two bf16 operands: half a step (2^-8) of half a step
    2^-20     2^x (or the quotient of SiLU) and the fp32 sums
    1.5e-4    of a Phi(-a) = max(x, 0) - GELU(x), a = |x|, by the polynomial of degree 8
    and what the scores' errors do to the weights, in the numerator and in the sum.  q has one column, so a
    score is q (s (c - 8) + z) in 6 roundings of its parts' size at most (2^-24 each)

With P s in one operand (2^-8), or a Phi that is right to 1.9e-3 (degree 6, where that errs most), the same
norm is above that, which restatements on the CPU show for every case here.
"""

import math

import numpy as np
import pytest
import torch

from oracle import step as oracle
from tests.test_cache4 import Case

gpu = pytest.mark.gpu


@pytest.fixture(scope="module")
def jg():
    from jagged_gdpa_gb300 import build as b
    b.build()
    import jagged_gdpa_gb300 as m
    return m


class Peaked(Case):
    """Scores by the queries' first column alone, all values above zero.  Softmax: every `every`th
    key around zero, the others some `spread` below.  SiLU: scores above zero, around `spread`.  GELU:
    scores near `spread`."""

    def __init__(self, ctx, new, d, act, spread, every, group=2):
        super().__init__(1, ctx, new, 2, group, d, 16, act, stale=False)
        rng = np.random.default_rng(1)
        self.scale = 1.0
        self.q.zero_()
        self.q[:, :, 0] = 1.0 + torch.from_numpy(rng.integers(0, 64, self.q.shape[:2])) / 128
        _, ks, vc, vs = self.cache
        if act == "gelu":
            self.q[:, :, 0] = 1.0
        ks[..., 0] = torch.from_numpy(rng.uniform(0.02, 0.06, ks.shape[:3]) / (1 if act != "gelu" else 5))
        at = rng.uniform(-0.5, 0.5, ks.shape[:3]) if act == "softmax" else spread * rng.uniform(0.7, 1.5, ks.shape[:3])
        if act == "softmax":
            at -= spread * (rng.integers(0, every, at.shape) > 0)
        elif act == "gelu":
            at = spread + rng.uniform(-0.1, 0.1, ks.shape[:3])
        ks[..., 1] = torch.from_numpy(at)
        vc.copy_(torch.from_numpy(oracle.pack(rng.integers(9, 16, (*vc.shape[:3], d))).copy()))
        vs[..., 1] = 0

    def rows(self, kernels):
        """(the definition's outputs, what x may be off by, and outputs of kernels that hold P s in so many
        bf16 operands and multiply GELU's weights by so much, all else exact)"""
        shape = (self.off[-1], self.heads, self.d)
        want, off, held = np.zeros(shape), np.zeros(shape), [np.zeros(shape) for _ in kernels]
        kc, ks, vc, vs = (t.double().numpy() for t in self.cache)
        k, codes = oracle.unpack(kc.astype(np.uint8)[..., :1])[..., 0] - 8, oracle.unpack(vc.astype(np.uint8)) - 8
        q = self.q.double().numpy()[..., 0]
        for b in range(len(self.new)):
            for t in range(self.new[b]):
                j = np.arange(self.kv[b] - self.new[b] + t + 1)
                page, place = self.table[b, j // 16], j % 16
                for h in range(self.heads):
                    at, r = (page, h // (self.heads // self.kv_heads), place), self.off[b] + t
                    step, middle, v = ks[at][:, 0], ks[at][:, 1], codes[at]
                    s = q[r, h] * (step * k[at] + middle)
                    es = 6 * 2.0 ** -24 * q[r, h] * (8 * step + np.abs(middle))
                    if self.act == "softmax":
                        p = np.exp(s - s.max())
                        p /= p.sum()
                        es = p * (es + (p * es).sum())
                    elif self.act == "silu":
                        p = s / (1 + np.exp(-s))
                        es = 1.1 * es  # |silu'| <= 1.1
                    else:
                        below = np.abs(s) * tail(np.abs(s))
                        p = np.maximum(s, 0) - below
                        # |gelu'| is 1.13 at most, and below zero Phi(-a) + a phi(a)
                        slope = np.where(s > 0, 1.13, tail(np.abs(s)) + np.abs(s) * np.exp(-s * s / 2) * 0.4)
                        es = slope * es + 1.5e-4 * below
                    y = p * vs[at][:, 0]
                    want[r, h] = y @ v
                    off[r, h] = np.abs(want[r, h]) * (2.0 ** -16 + 2.0 ** -20) + (es * vs[at][:, 0]) @ v
                    if self.act == "softmax":  # (as the kernel holds P, with its largest 1)
                        y = y / p.max()
                    for (n, wrong), out in zip(kernels, held):
                        taken, z = np.zeros_like(y), y if wrong is None else y * wrong(np.abs(s))
                        for _ in range(n):
                            taken += oracle.bf16((z - taken).astype(np.float32)).astype(np.float64)
                        out[r, h] = taken @ v * (p.max() if self.act == "softmax" else 1.0)
        return want, off, [rounded(x) for x in held]


def tail(a):
    """Phi(-a)"""
    return np.array([0.5 * math.erfc(x / math.sqrt(2)) for x in a])


def sixth(a):
    """What a polynomial of degree 6 for log2 Phi(-a), right to 1.9e-3, makes of Phi(-a), over Phi(-a)."""
    c = (3.53243581e-06, -0.000168592655, 0.0033006093, -0.0349358097, -0.492554843, -1.1279366, -1.00261784)
    return np.exp2(np.polyval(c, a)) / tail(a)


def rounded(x):
    return oracle.bf16(x.astype(np.float32)).astype(np.float64)


def ratio(got, want, off):
    """The norm of the outputs' errors and its bound, in units of what one rounding leaves."""
    r = np.linalg.norm(rounded(want) - want)
    return np.linalg.norm(got - want) / r, 1 + 2 * np.linalg.norm(off) / r


# (act, spread, every, context, new tokens): lengths on both sides of a block's 32 and a tile's 64 keys, of 256, and
# prompts without context, whose first rows see one key, two, three
CASES = [("softmax", 0.0, 1, [1, 2, 3, 1, 2, 3] * 4, [1] * 24), ("softmax", 10.0, 16, [39, 40, 62, 63, 64, 65] * 2, [1] * 12),
         ("softmax", 12.0, 80, [254, 255, 256, 299, 300] * 3, [1] * 15), ("softmax", 16.0, 1200, [4000, 3999] * 4, [1] * 8),
         ("softmax", 9.0, 30, [0, 0], [100, 70]), ("softmax", 12.0, 90, [0], [300]),
         ("silu", 3.0, 1, [0] * 8, [1] * 8), ("silu", 1.0, 1, [0, 1, 2] * 4, [1] * 12), ("silu", 2.0, 1, [0] * 12, [2, 5] * 6),
         ("gelu", 2.0, 1, [0] * 12, [1] * 12), ("gelu", -2.1, 1, [0, 1] * 6, [1] * 12), ("gelu", -4.5, 1, [0] * 12, [1] * 12),
         ("gelu", -2.1, 1, [199, 300], [1, 1]), ("gelu", -4.6, 1, [300], [3])]


@pytest.mark.parametrize("act,spread,every,ctx,new", CASES)
def test_one_operand_would_show(act, spread, every, ctx, new):
    kernels = [(2, None), (1, None), (2, sixth)][:3 if act == "gelu" and spread < 0 else 2]
    want, off, (good, *bad) = Peaked(ctx, new, 32, act, spread, every).rows(kernels)
    errors, bound = [ratio(x, want, off)[0] for x in bad], ratio(good, want, off)[1]
    assert ratio(good, want, off)[0] < bound
    # (over hundreds of keys one operand's errors average out)
    assert max(errors) > bound if act == "gelu" and max(ctx) > 10 else all(e > bound for e in errors)


@gpu
@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("group", [2, 12])
@pytest.mark.parametrize("act,spread,every,ctx,new", CASES)
def test_few_keys_carry_the_weight(jg, act, spread, every, ctx, new, group, d):
    c = Peaked(ctx, new, d, act, spread, every, group)
    want, off, _ = c.rows(())
    out, _ = jg.jgdpa_cache4_fwd(**c.kwargs())
    a, bound = ratio(out.double().cpu().numpy(), want, off)
    assert a <= bound
