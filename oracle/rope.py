"""Float64 CPU oracle for rotary positions.

TEST INFRASTRUCTURE ONLY, sharing no code with the CUDA library: pair by pair, the
products of bf16 and fp32 numbers exact in 64 bits, each result rounded once to bf16.
"""
from __future__ import annotations

import numpy as np
import torch


def round_bf16(x):
    """float64 values rounded to bf16's nearest, ties to even (float64 out)."""
    x = np.asarray(x, dtype=np.float64)
    with np.errstate(all="ignore"):
        _, e = np.frexp(x)
        step = np.ldexp(1.0, np.maximum(e.astype(np.int64) - 8, -133))
        y = np.round(x / step) * step
        y = np.where(np.abs(y) > 3.3895313892515355e38, np.copysign(np.inf, x), y)
    return np.where(np.isfinite(x), y, x)


def _sum_to_odd(p, q):
    """p + q cut off to float64, its last bit set where bits were lost: rounding
    that to fewer bits is rounding the sum itself, once."""
    with np.errstate(all="ignore"):
        h = p + q
        z = h - p
        rest = (p - (h - z)) + (q - z)
        lost = np.isfinite(h) & (rest != 0)
    bits = h.view(np.int64)
    return np.where(lost, (bits - ((rest < 0) != (h < 0))) | 1, bits).view(np.float64)


def rotate(x, positions, table, interleaved=False, transposed=False):
    """x [..., d] (float64), positions of x's shape without the last axis (or
    one that broadcasts), table [L, rot / 2, 2]: float64, not rounded
    to fewer bits.  Rows at positions outside the table pass."""
    x, table = np.asarray(x, dtype=np.float64), np.asarray(table, dtype=np.float64)
    L, half, _ = table.shape
    pos = np.broadcast_to(np.asarray(positions), x.shape[:-1])
    y = x.copy()
    for at in np.ndindex(*pos.shape):
        p = int(pos[at])
        if p < 0 or p >= L:
            continue
        c, s = table[p, :, 0], table[p, :, 1] * (-1 if transposed else 1)
        row = x[at]
        a, b = (row[0:2 * half:2], row[1:2 * half:2]) if interleaved else (row[:half], row[half:2 * half])
        with np.errstate(invalid="ignore"):
            re, im = _sum_to_odd(a * c, -(b * s)), _sum_to_odd(b * c, a * s)
        if interleaved:
            y[at][0:2 * half:2], y[at][1:2 * half:2] = re, im
        else:
            y[at][:half], y[at][half:2 * half] = re, im
    return y


def rope(x, positions, table, interleaved=False, transposed=False):
    """The same of a bf16 tensor, rounded to one."""
    x = x.detach().cpu()
    y = rotate(x.double().numpy(), positions, table.cpu().numpy(), interleaved, transposed)
    return torch.from_numpy(round_bf16(y)).to(torch.bfloat16)
