"""The oracle of rotary positions against exact rationals: every result is the
exact value rounded once."""
import math
from fractions import Fraction

import numpy as np
import torch

import oracle


def round_once(v: Fraction) -> float:
    """To bf16, nearest even."""
    if v == 0:
        return 0.0
    a = abs(v)
    e = a.numerator.bit_length() - a.denominator.bit_length()
    e = e if a >= Fraction(2) ** e else e - 1                    # 2^e <= a < 2^(e + 1)
    step = Fraction(2) ** max(e - 7, -133)
    r = round(a / step) * step                                   # round() of a Fraction: nearest even
    r = math.inf if r >= Fraction(2) ** 128 else float(r)
    return math.copysign(r, v)


def check(a, b, c, s):
    """Arrays of one pair each, a and b bf16 values, c and s fp32 ones."""
    n = len(a)
    for lo in range(0, n, 8):
        k = min(8, n - lo)
        x, table = np.zeros((1, 16)), np.zeros((1, 8, 2))
        x[0, :k], x[0, 8:8 + k] = a[lo:lo + k], b[lo:lo + k]
        table[0, :k, 0], table[0, :k, 1] = c[lo:lo + k], s[lo:lo + k]
        got = oracle.rope(torch.from_numpy(x).to(torch.bfloat16), [0], torch.from_numpy(table)).double().numpy()
        for i in range(k):
            A, B, C, S = (Fraction(float(v[lo + i])) for v in (a, b, c, s))
            assert got[0, i] == round_once(A * C - B * S), (lo + i, "first")
            assert got[0, 8 + i] == round_once(B * C + A * S), (lo + i, "second")


def test_round_once():
    x = torch.randn(500, generator=torch.Generator().manual_seed(1)).double() * 2.0 ** torch.arange(-140, 110).repeat(2)
    assert [round_once(Fraction(v)) for v in x.float().tolist()] == x.float().to(torch.bfloat16).tolist()
    assert round_once(Fraction(1) + Fraction(1, 256) + Fraction(1, 2 ** 200)) == 1.0078125


def test_ordinary_pairs():
    g = np.random.default_rng(2)
    a, b = (torch.from_numpy(g.normal(size=400) * 2.0 ** g.integers(-8, 8, 400)).to(torch.bfloat16).double().numpy()
            for _ in range(2))
    t = g.uniform(0, 6.3, 400)
    check(a, b, np.cos(t).astype(np.float32), np.sin(t).astype(np.float32))


def test_ties_decided_by_a_term_far_below():
    """64 bits hold neither sum: 1 + 2^-8 is a tie of bf16, the other term tells."""
    k = [1.0, 1.0, 1.0, 1.0, 2.0 ** -100, -2.0 ** -100, 2.0 ** -133, 2.0 ** -133]
    check(np.array([1.0, -1.0] * 4), np.array(k), np.full(8, 257 / 256, np.float32),
          np.array([2.0 ** -60, -2.0 ** -60, 2.0 ** -149, 2.0 ** -52] * 2, np.float32))


def test_small_numbers():
    g = np.random.default_rng(3)
    a, b = (torch.from_numpy(g.normal(size=200) * 2.0 ** g.integers(-133, -118, 200)).to(torch.bfloat16).double().numpy()
            for _ in range(2))
    t = g.uniform(0, 6.3, 200)
    check(a, b, np.cos(t).astype(np.float32), np.sin(t).astype(np.float32))
