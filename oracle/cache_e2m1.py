"""Float64 CPU oracle for the 4-bit key/value cache.

TEST INFRASTRUCTURE ONLY, sharing no code with the CUDA library: codes and
scales by comparison with the borders between them, bytes one by one, attention
row by row in float64 over the values.
"""
from __future__ import annotations

import math

import numpy as np
import torch

from .fp8 import e4m3_decode, e4m3_encode

MAGNITUDES = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])


def e2m1_encode(y):
    """The code nearest to each value, ties to the one with an even last bit."""
    y = np.asarray(y, dtype=np.float64)
    a = np.minimum(np.abs(y), 6.0)
    gap = np.abs(a[..., None] - MAGNITUDES)
    best = gap.min(-1, keepdims=True)
    near = gap == best
    even = near & (np.arange(8) % 2 == 0)
    code = np.where(even.any(-1), even.argmax(-1), near.argmax(-1))
    return (code + 8 * np.signbit(y)).astype(np.uint8)


def e2m1_decode(c):
    c = np.asarray(c)
    return MAGNITUDES[c & 7] * np.where(c & 8, -1.0, 1.0)


def quantise(x, unit):
    """Codes [.., d] and scale codes [.., d / 16] of x [.., d]."""
    x = np.asarray(x, dtype=np.float64)
    y = x.reshape(*x.shape[:-1], -1, 16) / unit
    s8 = e4m3_encode(np.minimum(np.abs(y).max(-1) / 6, 448.0))
    s = e4m3_decode(s8)[..., None]
    q = np.divide(y, s, out=np.zeros_like(y), where=s > 0)
    q = np.where(s > 0, q, np.copysign(0.0, y))
    return e2m1_encode(q).reshape(x.shape), s8


def places(d):
    """Of (token of 16, element): byte and shift of its code and byte of its
    scale, for K and for V."""
    out = []
    for is_v in (False, True):
        byte, shift, scale = (np.zeros((16, d), dtype=np.int64) for _ in range(3))
        for t in range(16):
            for e in range(d):
                g = e // 16
                if not is_v:
                    at = [0, 4, 1, 5, 2, 6, 3, 7].index(g) if d == 128 else g
                    byte[t, e] = t * d // 2 + at * 8 + e % 16 // 2
                    scale[t, e] = 8 * d + t * d // 16 + at
                else:
                    p = e // (d // 8)
                    swapped = p in (1, 3, 5, 7) if d == 128 else p in (2, 3, 6, 7)
                    where = (t + 8) % 16 if swapped else t
                    byte[t, e] = 9 * d + p * d + where * d // 16 + e % (d // 8) // 2
                    scale[t, e] = 17 * d + g * 16 + [0, 1, 8, 9, 2, 3, 10, 11, 4, 5, 12, 13, 6, 7, 14, 15].index(t)
                shift[t, e] = 4 * (e % 2)
        out.append((byte, shift, scale))
    return out


def append(data, k, v, slots, k_unit, v_unit):
    """Rows k, v [T, H, d] into data (numpy uint8 [blocks, H, P / 16, 18 d]), changed in place."""
    d = data.shape[3] // 18
    n = data.shape[2]
    where = places(d)
    for x, (byte, shift, scale), unit in ((k, where[0], k_unit), (v, where[1], v_unit)):
        code, s8 = quantise(x, unit)
        for t, s in enumerate(slots):
            if s < 0 or s >= data.shape[0] * 16 * n:
                continue
            row = data[s // (16 * n), :, s // 16 % n]
            tok = s % 16
            for h in range(data.shape[1]):
                c = code[t, h]
                row[h, byte[tok][0::2]] = c[0::2] | c[1::2] << 4
                row[h, scale[tok][::16]] = s8[t, h]


def values(data, k_unit, v_unit):
    """K and V of every token: float64 [blocks, H, P, d]."""
    d = data.shape[3] // 18
    out = []
    for (byte, shift, scale), unit in zip(places(d), (k_unit, v_unit)):
        x = e2m1_decode(data[..., byte] >> shift & 15) * e4m3_decode(data[..., scale]) * unit
        out.append(x.reshape(*data.shape[:2], 16 * data.shape[2], d))
    return out


def attention(q, data, k_unit, v_unit, table, seq_lens, cu, scale, causal=True):
    """O [T, Hq, d], L [T, Hq] (float64) and, per row, what the error bounds
    scale with: A = sum_j p_j |v_j|, S = the largest |scale| sum_t |q_t k_jt| over
    its visible keys, W = the largest p_j times sum_j |v_j|.  Rows of no request
    are NaN."""
    q = q.detach().to("cpu", torch.float64).numpy()
    table = np.asarray(table)
    T, Hq, d = q.shape
    H, P = data.shape[1], 16 * data.shape[2]
    g = Hq // H
    O, A, W = (np.full((T, Hq, d), np.nan) for _ in range(3))
    L, S = (np.full((T, Hq), np.nan) for _ in range(2))
    for r, N in enumerate(seq_lens):
        c0, n = cu[r], cu[r + 1] - cu[r]
        at = [int(b) for b in table[r][:-(-N // P)]]
        k, v = (x.transpose(0, 2, 1, 3).reshape(len(at) * P, H, d)[:N] for x in values(data[at], k_unit, v_unit))
        for i in range(n):
            seen = max(0, min(N, N - n + i + 1)) if causal else N
            for h in range(Hq):
                row = c0 + i, h
                if seen == 0:
                    O[row], A[row], W[row], L[row], S[row] = 0, 0, 0, -math.inf, 0
                    continue
                x, kh, vh = q[row], k[:seen, h // g], v[:seen, h // g]
                s = scale * (kh @ x)
                m = s.max()
                p = np.exp(s - m)
                L[row] = m + math.log(p.sum())
                p /= p.sum()
                O[row], A[row] = p @ vh, p @ np.abs(vh)
                S[row] = abs(scale) * (np.abs(kh) @ np.abs(x)).max()
                W[row] = p.max() * np.abs(vh).sum(0)
    return tuple(torch.from_numpy(a) for a in (O, L, A, S, W))
