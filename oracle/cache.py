"""Float64 CPU oracle for the 8-bit key/value cache.

TEST INFRASTRUCTURE ONLY, sharing no code with the CUDA library: slot
assignment request by request in Python integers, appends run by run, and
attention row by row in float64 over the dequantised cache.
"""
from __future__ import annotations

import math

import numpy as np
import torch

from .fp8 import e4m3_decode, e4m3_encode


def cache_slots(table, seq_lens, new_lens, free, used, P, num_tokens):
    """Lists and a list of rows in, the same out: (table, cu, slots, lens,
    used) after granting blocks in the order of the requests."""
    table = [list(row) for row in table]
    M = len(table[0]) if table else 0
    slots, cu, lens = [-1] * num_tokens, [0], []
    gone, asked = used, used  # asked also counts requests that did not get theirs
    for r, (n0, n) in enumerate(zip(seq_lens, new_lens)):
        n0, n = max(0, n0), max(0, n)
        start = cu[-1]
        cu.append(start + n)
        held, want = -(-n0 // P), -(-(n0 + n) // P)
        if want > M or start + n > num_tokens:
            lens.append(n0)
            continue
        need = want - held
        asked += need
        if need and asked > len(free):
            lens.append(n0)
            continue
        for j in range(need):
            table[r][held + j] = free[gone + j]
        gone += need
        lens.append(n0 + n)
        for i in range(n):
            b = table[r][(n0 + i) // P]
            slots[start + i] = b * P + (n0 + i) % P if b >= 0 else -1
    return table, cu, slots, lens, gone


def block_scale(a):
    """The smallest power of two s with a <= 448 s, its exponent within
    [-100, 120]."""
    e = -100
    while a > 448.0 * 2.0 ** e and e < 120:
        e += 1
    return 2.0 ** e


def cache_append(x, codes, scale, slots, P):
    """One of K and V: x [T, H, d] (values), codes uint8 [blocks, H, P, d] and
    scale float [blocks, H], changed in place (numpy)."""
    x = np.asarray(x, dtype=np.float64)
    T, t = len(slots), 0
    while t < T:
        s = int(slots[t])
        if s < 0 or s >= codes.shape[0] * P:
            t += 1
            continue
        n = 1
        while t + n < T and slots[t + n] == s + n and (s + n) % P != 0:
            n += 1
        b, off = divmod(s, P)
        for h in range(codes.shape[1]):
            part = x[t:t + n, h]
            now = block_scale(np.abs(part).max())
            if off > 0:
                old = float(scale[b, h])
                now = max(old, now)
                if now > old:
                    codes[b, h, :off] = e4m3_encode(e4m3_decode(codes[b, h, :off]) * (old / now))
            scale[b, h] = now
            codes[b, h, off:off + n] = e4m3_encode(part / now)
        t += n


def cache_values(codes, scale, table_row, n):
    """The n cached values [n, H, d] of one request (float64)."""
    P = codes.shape[2]
    at = [int(b) for b in table_row[:-(-n // P)]]
    v = e4m3_decode(codes[at]) * np.asarray(scale[at], dtype=np.float64)[:, :, None, None]
    return v.transpose(0, 2, 1, 3).reshape(len(at) * P, codes.shape[1], codes.shape[3])[:n]


def attention_cache(q, k8, v8, k_scale, v_scale, table, seq_lens, cu, scale, causal=True):
    """O [T, Hq, d], L [T, Hq] (float64) and, per row, what the error bounds
    scale with: A = sum_j p_j |v_j| [T, Hq, d], S = the largest
    |scale| sum_t |q_t k_jt| over its visible keys [T, Hq], R = the largest
    |scale| max |q| sum |k_jt| over the t with |q_t| < 2^-9 max |q| [T, Hq], and
    W = the largest p_j times its V scale, times the sum of |V code values|
    [T, Hq, d].  Rows of no request are NaN."""
    q = q.detach().to("cpu", torch.float64).numpy()
    k8, v8 = np.asarray(k8), np.asarray(v8)
    k_scale, v_scale, table = np.asarray(k_scale), np.asarray(v_scale), np.asarray(table)
    T, Hq, d = q.shape
    g = Hq // k8.shape[1]
    P = k8.shape[2]
    O, A, W = (np.full((T, Hq, d), np.nan) for _ in range(3))
    L, S, R = (np.full((T, Hq), np.nan) for _ in range(3))
    for r, n_keys in enumerate(seq_lens):
        c0, n = cu[r], cu[r + 1] - cu[r]
        k = cache_values(k8, k_scale, table[r], n_keys)
        v = cache_values(v8, v_scale, table[r], n_keys)
        v_unit = cache_values(v8, np.ones_like(v_scale), table[r], n_keys)
        v_size = v_scale[[int(table[r][j // P]) for j in range(n_keys)]].astype(np.float64).reshape(n_keys, k8.shape[1])
        for i in range(n):
            seen = max(0, min(n_keys, n_keys - n + i + 1)) if causal else n_keys
            for h in range(Hq):
                if seen == 0:
                    O[c0 + i, h], A[c0 + i, h], W[c0 + i, h], L[c0 + i, h] = 0, 0, 0, -math.inf
                    S[c0 + i, h], R[c0 + i, h] = 0, 0
                    continue
                x, kh, vh = q[c0 + i, h], k[:seen, h // g], v[:seen, h // g]
                s = scale * (kh @ x)
                m = s.max()
                p = np.exp(s - m)
                L[c0 + i, h] = m + math.log(p.sum())
                p /= p.sum()
                O[c0 + i, h], A[c0 + i, h] = p @ vh, p @ np.abs(vh)
                S[c0 + i, h] = abs(scale) * (np.abs(kh) @ np.abs(x)).max()
                small = np.abs(x) < 2.0 ** -9 * np.abs(x).max()
                R[c0 + i, h] = abs(scale) * np.abs(x).max() * np.abs(kh[:, small]).sum(1).max()
                W[c0 + i, h] = (p * v_size[:seen, h // g]).max() * np.abs(v_unit[:seen, h // g]).sum(0)
    return tuple(torch.from_numpy(a) for a in (O, L, A, S, R, W))
