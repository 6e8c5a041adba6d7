"""Inputs and bounds shared by the tests of the 8-bit key/value cache."""
import torch

import oracle

E4M3_MAX = 448.0


def make_tables(lens, P, extra_cols=1, spare=3, seed=0):
    """Distinct blocks in no order for requests of these lengths: (table int32
    [R, M], -1 behind a request's own, and the number of blocks)."""
    g = torch.Generator().manual_seed(seed)
    want = [-(-n // P) for n in lens]
    blocks = sum(want) + spare
    perm = torch.randperm(blocks, generator=g).tolist()
    M = max([1] + want) + extra_cols
    table, at = [], 0
    for w in want:
        table.append(perm[at:at + w] + [-1] * (M - w))
        at += w
    return torch.tensor(table, dtype=torch.int32).reshape(len(lens), M), blocks


def make_codes(blocks, H, P, d, seed, low=-6, high=-2):
    """Random codes (no NaN) and power-of-two scales 2^low .. 2^high."""
    g = torch.Generator().manual_seed(seed)
    c = torch.randint(0, 256, (blocks, H, P, d), generator=g, dtype=torch.int32)
    c = torch.where((c & 0x7F) == 0x7F, c - 0x10, c)
    # values spread like a rounded tensor's rather than over all exponents
    c = torch.where((c & 0x7F) < 0x30, c | 0x30, c)
    e = torch.randint(low, high + 1, (blocks, H), generator=g)
    return c.to(torch.uint8), torch.exp2(e.to(torch.float32)) / 16


def poison(codes, table, lens):
    """NaN codes behind each request's last token, and in every block of none."""
    P = codes.shape[2]
    used = set()
    for r, n in enumerate(lens):
        for j in range(-(-n // P)):
            b = int(table[r, j])
            used.add(b)
            if (j + 1) * P > n:
                codes[b, :, n - j * P:] = 0x7F
    for b in range(codes.shape[0]):
        if b not in used:
            codes[b] = 0xFF


def forward_bounds(O, L, A, S, R, W, d):
    """Element-wise bounds of |O - o| and |L - l| (float64 oracle values).

    Score of one key, in natural units, with u = 2^-24 (fp32): the fp32 sum of
    d products moves it by at most (d + 2) u S (S = the largest sum of
    |terms|); the row's exponent, the block's scale and scale * log2(e) are
    four more roundings, and the reference's subtraction one of the reduced
    score: 6 u S.  Query elements below 2^-17 of the row's largest lose up to
    2^-25 of it each, below 2 u S as the largest itself may meet a key element
    of zero: counted with d u S.  With many rows the query is two E4M3 numbers
    an element, its largest in [2^7, 2^8): elements of 2^-2 and more (8
    significant bits, the lowest of them 2^-9 or more) are exact, 4 bits of
    them in the first number and the rest, at most 8 steps of the lowest bit,
    in the second; smaller ones are rounded to 2^-9, off by 2^-10, 2^-17 of the
    largest: 2^-17 R (R: over the elements below 2^-9 of the largest).
    Together delta = (2 d + 8) u S + 2^-17 R, and 2^x (relative error 2^-22)
    makes it eps = delta + 2^-21 of a weight.
    O: weights carry eps in the numerator, eps in the sum, and the f16
    rounding of a weight, half of 2^-10 relative; the sums and divisions below
    2^-18 in all; then bf16, half of 2^-7 of the result.  A weight times its V
    scale is at most w = max p_j scale_j and is rounded as 2^14 times a number
    in which w lies in [1, 2), or with many rows as 2^10 times one in which it
    lies in [1, 2^5): below f16's smallest normal number its rounding is off by
    up to half of f16's smallest step, 2^-25, that is by 2^-35 w, and moves the
    result by 2^-35 w |V code value| for that key: 2^-35 W in all (which counts
    where the heaviest keys are 0 in a column).
    L: eps, the logarithm's and the last product's rounding."""
    u = 2.0 ** -24
    eps = (2 * d + 8) * u * S + 2.0 ** -17 * R + 2.0 ** -21
    bO = (2 * eps[..., None] + 2.0 ** -11 + 2.0 ** -18) * A + 2.0 ** -35 * W
    bO = bO + 2.0 ** -8 * (O.abs() + bO) + 1e-30
    bL = eps + 2.0 ** -20 + 4 * u * L.abs()
    return bO, bL


def assert_forward(o, lse, q, codes, table, lens, cu, scale, causal, what=""):
    """o, lse (any device) against the oracle on the rows of requests; returns
    the worst share of the bounds that was used."""
    k8, v8, ks, vs = codes
    O, L, A, S, R, W = oracle.attention_cache(q, k8.numpy(), v8.numpy(), ks.numpy(), vs.numpy(), table.numpy(), lens, cu,
                                        scale, causal)
    o, lse = o.detach().to("cpu", torch.float64), lse.detach().to("cpu", torch.float64)
    real = ~torch.isnan(L)
    empty = torch.isinf(L)
    assert torch.equal(lse[empty], L[empty]), f"{what}: L of rows without keys"
    assert (o[empty] == 0).all(), f"{what}: O of rows without keys"
    live = real & ~empty
    bO, bL = forward_bounds(O, L, A, S, R, W, q.shape[-1])
    assert torch.isfinite(o[live]).all() and torch.isfinite(lse[live]).all(), f"{what}: not finite"
    if not live.any():
        return 0.0
    rO = ((o - O).abs() / bO)[live].max().item()
    rL = ((lse - L).abs() / bL)[live].max().item()
    assert rO <= 1 and rL <= 1, f"{what}: |dO|/bound {rO:.3f}, |dL|/bound {rL:.3f}"
    return max(rO, rL)
