"""A call on many tokens gives a thread several rows, a call on few one: the same bits,
also where the rows do not divide by a thread's, or run from K into V."""
import pytest
import torch

import exact_attention_forward_04_gb300 as fa

pytestmark = pytest.mark.gpu

DEV = "cuda"


def _rows(T, H, d, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randn(T, H, d, generator=g, device=DEV).to(torch.bfloat16)


@pytest.mark.parametrize("d", (64, 128))
@pytest.mark.parametrize("H,T", ((5, 6000), (5, 14000), (3, 40000), (11, 20000), (1, 60000)))
def test_append_and_read(d, H, T):
    T = T * 128 // d
    P, few = 64, 700
    k, v = _rows(T, H, d, 1), _rows(T, H, d, 2)
    table, pos = fa.rope_table(1000, d - 16), (torch.arange(T, device=DEV) % 1003 - 2).int()
    pos[pos >= 1000] = -1
    slots = torch.randperm(T, device=DEV, generator=torch.Generator(device=DEV).manual_seed(3))
    for kw in ({}, dict(positions=pos, table=table), dict(positions=pos, table=table, interleaved=True)):
        one, two = (fa.cache_alloc_e2m1(T // P + 1, H, P, d, 0.25, 0.5) for _ in range(2))
        fa.cache_append_e2m1(k, v, one, slots, **kw)
        for i in range(0, T, few):
            part = {n: x[i:i + few] if n == "positions" else x for n, x in kw.items()}
            fa.cache_append_e2m1(k[i:i + few], v[i:i + few], two, slots[i:i + few], **part)
        assert torch.equal(one.data, two.data)
    together = fa.cache_read_e2m1(one, slots)
    parts = [fa.cache_read_e2m1(one, slots[i:i + few]) for i in range(0, T, few)]
    fa.check_errors()
    for i in (0, 1):
        assert torch.equal(together[i], torch.cat([p[i] for p in parts]))


@pytest.mark.parametrize("d", (64, 128))
@pytest.mark.parametrize("H,T", ((5, 8000), (7, 16000), (21, 20000), (37, 20000)))
def test_rope(d, H, T):
    T, few = T * 128 // d, 400
    x, table = _rows(T, H, d, 4), fa.rope_table(1000, d // 2)
    pos = (torch.arange(T, device=DEV) * 7 % 1000).int()
    for interleaved in (False, True):
        y = fa.rope(x, pos, table, interleaved=interleaved)
        parts = [fa.rope(x[i:i + few], pos[i:i + few], table, interleaved=interleaved) for i in range(0, T, few)]
        assert torch.equal(y, torch.cat(parts))
        z = x.clone()
        assert torch.equal(fa.rope(z, pos, table, interleaved=interleaved, out=z), y)
    fa.check_errors()
