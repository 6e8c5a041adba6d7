"""Inputs and bounds shared by the tests of the 4-bit key/value cache."""
import torch

import oracle
from tests.cache_cases import forward_bounds


def make_data(blocks, H, P, d, seed, low=0x28, high=0x48):
    """Random codes, and random scale codes low .. high (E4M3: 2^-2 .. 4)."""
    g = torch.Generator().manual_seed(seed)
    data = torch.randint(0, 256, (blocks, H, P // 16, 18 * d), generator=g, dtype=torch.int32)
    scale = torch.randint(low, high + 1, data.shape, generator=g, dtype=torch.int32)
    at = torch.arange(18 * d)
    is_scale = ((at >= 8 * d) & (at < 9 * d)) | (at >= 17 * d)
    return torch.where(is_scale, scale, data).to(torch.uint8)


def poison(data, table, lens):
    """Scales that are no number behind each request's last token, and in every block of none."""
    d, P = data.shape[3] // 18, 16 * data.shape[2]
    (_, _, ks), (_, _, vs) = oracle.cache_e2m1.places(d)
    used = set()
    for r, n in enumerate(lens):
        for j in range(-(-n // P)):
            b = int(table[r, j])
            used.add(b)
            for t in range(max(0, n - j * P), P):
                for where in (ks, vs):
                    data[b, :, t // 16, torch.from_numpy(where[t % 16])] = 0x7F
    for b in range(data.shape[0]):
        if b not in used:
            data[b] = 0xFF


def assert_forward(o, lse, q, data, units, table, lens, cu, scale, causal, what=""):
    """o, lse (any device) against the oracle on the rows of requests; returns
    the worst share of the bounds that was used.

    The bounds are those of the 8-bit cache's forward (cache_cases.forward_bounds)
    with R = 0, as the queries are one f16 number an element in both kernels, and
    W = max p_j sum |v_j|: the values enter the product with V as they are (f16
    holds them) and a weight is 2^(14 + s - m), or with many rows 2^(10 + s - m)
    with m up to 2^4 below the largest, as there with scales of 1."""
    O, L, A, S, W = oracle.cache_e2m1.attention(q, data.numpy(), *units, table.numpy(), lens, cu, scale, causal)
    o, lse = o.detach().to("cpu", torch.float64), lse.detach().to("cpu", torch.float64)
    real, empty = ~torch.isnan(L), torch.isinf(L)
    assert torch.equal(lse[empty], L[empty]), f"{what}: L of rows without keys"
    assert (o[empty] == 0).all(), f"{what}: O of rows without keys"
    live = real & ~empty
    if not live.any():
        return 0.0
    bO, bL = forward_bounds(O, L, A, S, torch.zeros_like(S), W, q.shape[-1])
    assert torch.isfinite(o[live]).all() and torch.isfinite(lse[live]).all(), f"{what}: not finite"
    rO = ((o - O).abs() / bO)[live].max().item()
    rL = ((lse - L).abs() / bL)[live].max().item()
    assert rO <= 1 and rL <= 1, f"{what}: |dO|/bound {rO:.3f}, |dL|/bound {rL:.3f}"
    return max(rO, rL)
