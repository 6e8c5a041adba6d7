"""The 4-bit key/value cache on the GPU against the float64 oracle: appended
bytes exactly, attention within derived bounds (``cache4_cases.assert_forward``)."""
import math

import numpy as np
import pytest
import torch

import exact_attention_forward_04_gb300 as fa
import oracle
from tests.cache4_cases import assert_forward, make_data, poison
from tests.cache_cases import make_tables

pytestmark = pytest.mark.gpu

DEV = "cuda"


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _rows(T, H, d, seed, low=-6, high=6):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, H, d, generator=g) * torch.exp2(torch.randint(low, high + 1, (T, H, 1), generator=g).float())
    return x.to(torch.bfloat16).to(DEV)


def _cache(blocks, H, P, d, seed, k_unit=1.0, v_unit=1.0):
    return fa.CacheE2M1(make_data(blocks, H, P, d, seed).to(DEV), k_unit, v_unit)


def _codes_equal(got, want, what=""):
    """Bytes, where a zero's sign does not count."""
    got, want = got.cpu().numpy(), want
    d = got.shape[3] // 18
    bad = got != want
    if bad.any():
        at = np.arange(18 * d)
        scale = ((at >= 8 * d) & (at < 9 * d)) | (at >= 17 * d)
        no_sign = lambda x: (np.where(x & 7, x & 15, 0) | np.where(x >> 4 & 7, x & 0xF0, 0))  # noqa: E731
        bad &= ~(~scale & (no_sign(got) == no_sign(want)))
    assert not bad.any(), f"{what}: {int(bad.sum())} bytes differ, first at {np.argwhere(bad)[:3].tolist()}"


# ------------------------------------------------------------------ append

def _append_case(slots, H, P, d, blocks, rot=0, interleaved=False, k_unit=1.0, v_unit=1.0, seed=0, k=None, v=None):
    T = len(slots)
    k = _rows(T, H, d, seed + 1) if k is None else k
    v = _rows(T, H, d, seed + 2) if v is None else v
    cache = _cache(blocks, H, P, d, seed + 3, k_unit, v_unit)
    ref = cache.data.cpu().numpy().copy()
    kw, kr = {}, k.cpu()
    if rot:
        g = torch.Generator().manual_seed(seed)
        pos = torch.randint(-1, 700, (T,), generator=g, dtype=torch.int32)
        kw = dict(positions=pos.to(DEV), table=fa.rope_table(700, rot), interleaved=interleaved)
        kr = oracle.rope(k, pos[:, None].numpy(), kw["table"], interleaved)
    sl = torch.tensor(slots, dtype=torch.int64, device=DEV)
    fa.cache_append_e2m1(k, v, cache, sl, **kw)
    fa.check_errors()
    oracle.cache_e2m1.append(ref, kr.double().numpy(), v.cpu().double().numpy(), slots, k_unit, v_unit)
    _codes_equal(cache.data, ref, f"P={P} d={d} H={H} rot={rot}")
    return cache, sl, kw, k, v


@pytest.mark.parametrize("P", (16, 32, 64, 128))
@pytest.mark.parametrize("d", (64, 128))
@pytest.mark.parametrize("H,T", ((1, 1), (3, 50), (8, 300)))
def test_append(P, d, H, T):
    """Slots in any order, some skipped; a few rows to many."""
    g = torch.Generator().manual_seed(T + P)
    blocks = T // P + 3
    slots = torch.randperm(blocks * P, generator=g)[:T].tolist()
    slots[::7] = [-1] * len(slots[::7]) if T > 1 else slots[::7]
    _append_case(slots, H, P, d, blocks, seed=P)


@pytest.mark.parametrize("interleaved", (False, True))
@pytest.mark.parametrize("d,rot", [(64, r) for r in (16, 32, 48, 64)] + [(128, r) for r in (16, 48, 64, 96, 128)])
def test_append_turned(d, rot, interleaved):
    """K turned on the way is K turned before, to the bit; V is not turned."""
    T, H, P = 75, 3, 32
    slots = torch.randperm(4 * P, generator=torch.Generator().manual_seed(rot))[:T].tolist()
    cache, sl, kw, k, v = _append_case(slots, H, P, d, 4, rot, interleaved, seed=rot)
    two = fa.CacheE2M1(make_data(4, H, P, d, rot + 3).to(DEV))
    fa.cache_append_e2m1(fa.rope(k, **{**kw}), v, two, sl)
    assert torch.equal(cache.data, two.data)


def test_append_many_heads_and_tokens():
    _append_case(list(range(40)), 40, 16, 64, 4, 64, False)
    _append_case(list(range(3000, 100, -1)), 5, 128, 128, 24, 128, True)


@pytest.mark.parametrize("k_unit,v_unit", ((2.0 ** -64, 2.0 ** 64), (2.0 ** -9, 0.25), (8.0, 2.0 ** -20)))
def test_append_units(k_unit, v_unit):
    slots = list(range(5, 45))
    k = (_rows(40, 2, 128, 1, -2, 2).float() * k_unit).to(torch.bfloat16)
    v = (_rows(40, 2, 128, 2, -2, 2).float() * v_unit).to(torch.bfloat16)
    _append_case(slots, 2, 64, 128, 2, k=k, v=v, k_unit=k_unit, v_unit=v_unit)


def test_append_every_border():
    """Every bf16 quotient of 8 bits against every scale's rounding: groups
    whose largest runs over the mantissas, the others over all borders, from below the
    smallest scale to above the largest."""
    m = torch.arange(128, 256).float() / 128                      # [1, 2)
    top = torch.cat([m * 2.0 ** e for e in range(-12, 14)])        # largest of a group
    frac = torch.cat([m * 2.0 ** e for e in range(-5, 1)])         # of it
    g = torch.Generator().manual_seed(1)
    x = top[:, None] * frac[torch.randint(0, frac.numel(), (top.numel(), 64), generator=g)] / 2
    x = x * torch.where(torch.rand(x.shape, generator=g) < 0.5, -1, 1)
    x[:, ::16] = top[:, None]
    ties = torch.tensor([.25, .75, 1.25, 1.75, 2.5, 3.5, 5.])
    x[:, 1:8] = top[:, None] / 6 * ties
    scale = torch.from_numpy(oracle.e4m3_decode(oracle.e4m3_encode((top / 6).clamp(max=448).double().numpy()))).float()
    x[:, 17:24] = (scale[:, None] * ties)                          # exactly on the border where bf16 holds it
    x = x.to(torch.bfloat16)[:, None].to(DEV)
    T = x.shape[0]
    _append_case(list(range(T)), 1, 128, 64, T // 128 + 1, k=x, v=-x)


def test_append_zeros_infinities_and_nan():
    k = torch.zeros(3, 1, 64, dtype=torch.bfloat16)
    k[0, 0, 3], k[1, 0, 20], k[1, 0, 21] = float("inf"), -float("inf"), 5.0
    k[2, 0, 40] = float("nan")
    k[2, 0, 0] = 3.0
    cache = fa.cache_alloc_e2m1(1, 1, 16, 64)
    sl = torch.arange(3, device=DEV)
    fa.cache_append_e2m1(k.to(DEV), k.to(DEV), cache, sl)
    for t in fa.cache_read_e2m1(cache, sl):
        assert t[0, 0, 3] == 6 * 448 and t[1, 0, 20] == -6 * 448
        assert (t[0, 0, 16:] == 0).all() and torch.isfinite(t).all()
        assert t[2, 0, 0] == 3 and (t[2, 0, 1:32] == 0).all() and (t[2, 0, 48:] == 0).all()
    fa.check_errors()


def test_append_strided_rows_and_slots_out_of_range():
    T, H, d, P = 30, 3, 64, 16
    kv = _rows(T, 2 * H + 1, d, 5)
    slots = list(range(T))
    _append_case(slots, H, P, d, 3, rot=32, k=kv[:, :H], v=kv[:, H:2 * H])
    cache = _cache(3, H, P, d, 1)
    ref = cache.data.cpu().numpy().copy()
    bad = [0, 48, -2, 5, -1, 2 ** 62]
    k, v = _rows(6, H, d, 7), _rows(6, H, d, 8)
    fa.cache_append_e2m1(k, v, cache, torch.tensor(bad, device=DEV))
    with pytest.raises(fa.FAError) as e:
        fa.check_errors()
    assert e.value.status == -6 and "site=601" in str(e.value)
    oracle.cache_e2m1.append(ref, k.cpu().double().numpy(), v.cpu().double().numpy(), bad, 1.0, 1.0)
    _codes_equal(cache.data, ref)
    pos, table = i32([0, 1, 2, 99, 1, 1]), fa.rope_table(50, 32)
    fa.cache_append_e2m1(k, v, cache, torch.tensor([0, 1, 2, 3, 4, 5], device=DEV), positions=pos, table=table)
    with pytest.raises(fa.FAError) as e:
        fa.check_errors()
    assert "site=621" in str(e.value)
    one, two = (fa.CacheE2M1(cache.data.clone()) for _ in range(2))  # the row beyond the table as it is
    sl = torch.tensor([7, 8], device=DEV)
    fa.cache_append_e2m1(k[:2], v[:2], one, sl, positions=i32([50, 3]), table=table)
    with pytest.raises(fa.FAError):
        fa.check_errors()
    fa.cache_append_e2m1(k[:2], v[:2], two, sl, positions=i32([-1, 3]), table=table)
    fa.check_errors()
    assert torch.equal(one.data, two.data)


def test_nothing():
    cache = fa.cache_alloc_e2m1(2, 2, 16, 64)
    none, no = torch.zeros(0, 2, 64, dtype=torch.bfloat16, device=DEV), torch.zeros(0, dtype=torch.int64, device=DEV)
    fa.cache_append_e2m1(none, none, cache, no)
    assert fa.cache_read_e2m1(cache, no)[0].shape == (0, 2, 64)
    o, lse = fa.cache_forward_e2m1(none, cache, i32([[0]]), i32([1]), i32([0, 0]))
    assert o.shape == (0, 2, 64) and lse.shape == (0, 2)
    fa.check_errors()
    assert (cache.data == 0).all()


@pytest.mark.parametrize("P,d,H", ((16, 64, 3), (128, 128, 2), (32, 128, 9)))
def test_read(P, d, H):
    cache = _cache(4, H, P, d, 3, 2.0 ** -30, 4.0)
    kk, vv = oracle.cache_e2m1.values(cache.data.cpu().numpy(), 2.0 ** -30, 4.0)
    slots = torch.randperm(4 * P, generator=torch.Generator().manual_seed(1))[:50].tolist() + [-1]
    k, v = fa.cache_read_e2m1(cache, torch.tensor(slots, device=DEV))
    fa.check_errors()
    for got, want in ((k, kk), (v, vv)):
        want = want.transpose(0, 2, 1, 3).reshape(4 * P, H, d)[slots[:-1]]
        assert np.array_equal(got.cpu().double().numpy()[:-1], want) and (got[-1] == 0).all()
    k, v = fa.cache_read_e2m1(cache, torch.tensor([3, 4 * P, -9], device=DEV))
    with pytest.raises(fa.FAError) as e:
        fa.check_errors()
    assert "site=631" in str(e.value)
    assert (k[1:] == 0).all() and (v[1:] == 0).all() and not (v[0] == 0).all()


# ----------------------------------------------------------------- forward

def _forward_case(lens, new, P, H, g, d, causal=True, scale=None, seed=0, sigma=1.0, units=(0.5, 2.0), spread=None, **kw):
    table, blocks = make_tables(lens, P, seed=seed)
    data = make_data(blocks, H, P, d, seed + 1, *(spread or ()))
    poison(data, table, lens)
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    gen = torch.Generator().manual_seed(seed + 3)
    q = (torch.randn(cu[-1] + 2, H * g, d, generator=gen) * sigma).to(torch.bfloat16)  # two rows of no request
    scale = 0.3 / math.sqrt(d) if scale is None else scale
    o, lse = fa.cache_forward_e2m1(q.to(DEV), fa.CacheE2M1(data.to(DEV), *units), table.to(DEV), i32(lens), i32(cu),
                                   scale=scale, causal=causal, **kw)
    fa.check_errors()
    what = f"lens={lens[:4]} new={new[:4]} P={P} H={H} g={g} d={d} causal={causal}"
    return assert_forward(o, lse, q, data, units, table, lens, cu, scale, causal, what)


@pytest.mark.parametrize("P", (16, 32, 64, 128))
@pytest.mark.parametrize("d", (64, 128))
@pytest.mark.parametrize("g", (1, 3, 8, 16))
def test_forward_decode(P, d, g):
    """Single tokens: lengths of one, around tiles and blocks, and longer ones."""
    lens = [1, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 129, 300, 777]
    _forward_case(lens, [1] * len(lens), P, 2, g, d, seed=g)


@pytest.mark.parametrize("d", (64, 128))
@pytest.mark.parametrize("causal", (True, False))
@pytest.mark.parametrize("g", (1, 4, 5))
def test_forward_drafts_and_prompts(d, causal, g):
    """Several tokens a request, none, more than it has cached, whole prompts."""
    lens, new = [40, 100, 0, 7, 3, 90, 0, 64], [3, 1, 2, 7, 5, 90, 0, 33]
    _forward_case(lens, new, 32, 2, g, d, causal=causal, seed=g)


@pytest.mark.parametrize("P", (16, 32, 64, 128))
@pytest.mark.parametrize("d", (64, 128))
@pytest.mark.parametrize("g", (1, 4, 7))
def test_forward_prompts(P, d, g):
    """Tens of rows and more per kv head: whole prompts and chunks behind a
    prefix, one half of a row tile and both, lengths around the key tiles."""
    lens, new = [127, 128, 129, 300, 40, 1, 260], [127, 60, 129, 33, 1, 1, 70]
    _forward_case(lens, new, P, 1, g, d, seed=g)


@pytest.mark.parametrize("d", (64, 128))
def test_forward_prompts_not_causal_and_other_scales(d):
    _forward_case([200, 90], [70, 90], 32, 2, 4, d, causal=False, seed=3)
    _forward_case([200, 90], [70, 90], 64, 1, 4, d, scale=-0.05, seed=4)
    _forward_case([200, 90], [70, 90], 16, 1, 4, d, scale=0.0, seed=5)
    _forward_case([200, 90], [1, 2], 16, 1, 4, d, scale=-0.05, seed=5)
    _forward_case([200, 90], [1, 2], 16, 1, 4, d, scale=0.0, seed=5)


@pytest.mark.parametrize("P", (16, 64))
def test_forward_prompt_behind_a_long_prefix(P):
    """Many key tiles, units split over CTAs, references that keep rising."""
    _forward_case([2600], [150], P, 2, 2, 64, sigma=4.0, seed=6)
    _forward_case([1900, 5], [40, 5], P, 1, 8, 128, sigma=6.0, seed=7)


def test_forward_prompts_longer_than_what_is_cached():
    _forward_case([5, 0, 130], [100, 40, 140], 32, 1, 4, 64, seed=8)


def test_forward_one_long_request():
    """One unit over all SMs, merged."""
    _forward_case([9001], [1], 64, 1, 4, 128, seed=2)
    _forward_case([5000], [2], 16, 2, 1, 64, seed=3)


def test_forward_many_requests():
    g = torch.Generator().manual_seed(8)
    lens = torch.randint(0, 40, (700,), generator=g).tolist()
    new = [min(n, int(x)) for n, x in zip(lens, torch.randint(0, 3, (700,), generator=g))]
    _forward_case(lens, new, 16, 1, 2, 64, seed=4)


def test_forward_wide_groups_and_heads():
    _forward_case([130, 50], [1, 1], 64, 1, 40, 128, seed=5)   # more rows than a tile
    _forward_case([70], [1], 32, 24, 1, 64, seed=6)


@pytest.mark.parametrize("d", (64, 128))
@pytest.mark.parametrize("new", (1, 40))
@pytest.mark.parametrize("units", ((2.0 ** -64, 2.0 ** -64), (2.0 ** 64, 2.0 ** 64), (2.0 ** -20, 2.0 ** 30)))
def test_forward_units(d, new, units):
    """The units are factors of the scale and of O, whatever their size."""
    _forward_case([100, 45], [new, new], 32, 2, 2, d, scale=0.04 / units[0], units=units)


@pytest.mark.parametrize("d", (64, 128))
@pytest.mark.parametrize("new", (1, 40))
def test_forward_scales_of_the_whole_range(d, new):
    """Scale codes from 0 (2^-9 steps) to 448 beside each other."""
    _forward_case([150, 77], [new, new], 32, 2, 2, d, scale=2.0 ** -12, spread=(0, 0x7E), seed=3)


@pytest.mark.parametrize("new", (1, 40))
def test_forward_peaky_rows(new):
    _forward_case([700, 333], [new, new], 64, 1, 4, 128, sigma=30.0, scale=0.3, seed=4)


@pytest.mark.parametrize("d", (64, 128))
@pytest.mark.parametrize("g,high", ((1, 1), (4, 2), (12, 2), (12, 30)))
def test_forward_many_pieces_the_same_every_time(d, g, high):
    """Many units of very different lengths a CTA: the same bits from every
    call, and right."""
    gen = torch.Generator().manual_seed(g + d)
    R, H, P = 160, 8, 16
    lens = (torch.randint(0, 40, (R,), generator=gen) ** 2).tolist()
    new = [min(n, int(x)) for n, x in zip(lens, torch.randint(0, high + 1, (R,), generator=gen))]
    table, blocks = make_tables(lens, P, seed=g)
    data = make_data(blocks, H, P, d, 1)
    poison(data, table, lens)
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    q = torch.randn(cu[-1], H * g, d, generator=gen).to(torch.bfloat16)
    args = (q.to(DEV), fa.CacheE2M1(data.to(DEV)), table.to(DEV), i32(lens), i32(cu), 0.3 * d ** -0.5)
    o, lse = fa.cache_forward_e2m1(*args)
    for _ in range(40):
        o2, lse2 = fa.cache_forward_e2m1(*args)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
    fa.check_errors()
    h = 5  # one kv head of the whole batch against the oracle
    at = slice(h * g, h * g + g)
    assert_forward(o[:, at], lse[:, at], q[:, at], data[:, h:h + 1], (1.0, 1.0), table, lens, cu, 0.3 * d ** -0.5, True,
                   f"d={d} g={g}")


@pytest.mark.parametrize("m", (120, 60, -60, -118, -130))
@pytest.mark.parametrize("new", (1, 40))
def test_forward_query_magnitudes(m, new):
    """Rows of any size, some elements far below their largest."""
    lens, P, H, g, d = [90, 50], 16, 1, 4, 64
    table, blocks = make_tables(lens, P, seed=m)
    data = make_data(blocks, H, P, d, 1)
    gen = torch.Generator().manual_seed(2)
    cu = [0, new, 2 * new]
    q = torch.randn(cu[-1], g, d, generator=gen, dtype=torch.float64) * 2.0 ** m
    q[:, :, ::5] *= 2.0 ** -12
    q = q.to(torch.bfloat16)
    scale = 2.0 ** (-m - 5) if -m - 5 < 127 else 2.0 ** 126
    o, lse = fa.cache_forward_e2m1(q.to(DEV), fa.CacheE2M1(data.to(DEV)), table.to(DEV), i32(lens), i32(cu), scale)
    fa.check_errors()
    assert_forward(o, lse, q, data, (1.0, 1.0), table, lens, cu, scale, True)


@pytest.mark.parametrize("d", (64, 128))
@pytest.mark.parametrize("g", (2, 5, 12, 34))
def test_forward_rows_that_are_not_finite(d, g):
    """An infinity or NaN in a query row spoils that row only."""
    lens, P, H = [300, 70], 16, 1
    table, blocks = make_tables(lens, P, seed=g)
    data = make_data(blocks, H, P, d, 1)
    q = torch.randn(2, H * g, d, generator=torch.Generator().manual_seed(g)).to(torch.bfloat16)
    bad = q.clone()
    bad[0, 1, 5], bad[1, 0, 7] = float("inf"), float("nan")
    cache, cu = fa.CacheE2M1(data.to(DEV)), i32([0, 1, 2])
    outs = [fa.cache_forward_e2m1(x.to(DEV), cache, table.to(DEV), i32(lens), cu, 0.04) for x in (q, bad)]
    fa.check_errors()
    keep = torch.ones(2, H * g, dtype=torch.bool)
    keep[0, 1] = keep[1, 0] = False
    for a, b in zip(*outs):
        assert torch.equal(a.cpu()[keep], b.cpu()[keep])


def test_forward_strided_queries_and_untouched_rows():
    lens, P, H, g, d = [100, 33], 32, 2, 2, 64
    table, blocks = make_tables(lens, P, seed=1)
    data = make_data(blocks, H, P, d, 2)
    wide = torch.randn(6, H * g + 3, d, generator=torch.Generator().manual_seed(4)).to(torch.bfloat16).to(DEV)
    q, cache, cu = wide[:, :H * g], fa.CacheE2M1(data.to(DEV)), i32([0, 2, 4])
    lib, size = fa.load_library(), fa.cache_forward_e2m1_workspace_size(2, 6, H * g, H, d)
    o = torch.full((6, H * g, d), 7.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((6, H * g), 7.0, device=DEV)
    ws = torch.empty(size, dtype=torch.uint8, device=DEV)
    t, sl = table.to(DEV), i32(lens)
    st = lib.fa_cache_fwd_e2m1(q.data_ptr(), q.stride(0), cache.data.data_ptr(), 1.0, 1.0, t.data_ptr(), sl.data_ptr(),
                               cu.data_ptr(), None, o.data_ptr(), lse.data_ptr(), 2, 6, H * g, H, d, blocks, P,
                               table.shape[1], 0.04, 1, ws.data_ptr(), size, torch.cuda.current_stream().cuda_stream)
    assert st == 0
    fa.check_errors()
    assert (o[4:] == 7).all() and (lse[4:] == 7).all()
    o2, lse2 = fa.cache_forward_e2m1(q.contiguous(), cache, t, sl, cu, 0.04, workspace=ws)
    assert torch.equal(o[:4], o2[:4]) and torch.equal(lse[:4], lse2[:4])
    assert_forward(o[:4], lse[:4], q[:4].cpu(), data, (1.0, 1.0), table, lens, [0, 2, 4], 0.04, True)


@pytest.mark.parametrize("P", (16, 64))
@pytest.mark.parametrize("new", (1, 40))
def test_forward_reports_what_is_out_of_range(P, new):
    """Blocks outside the cache hide their keys; lengths and rows are cut off."""
    lens, d = [6 * P + 4, 40], 64
    table, blocks = make_tables(lens, P, seed=1)
    data = make_data(blocks, 1, P, d, 2)
    q = torch.randn(2 * new, 1, d, generator=torch.Generator().manual_seed(4)).to(torch.bfloat16)
    cache, cu = fa.CacheE2M1(data.to(DEV)), [0, new, 2 * new]
    for entry in (blocks, -5, -1, 2 ** 31 - 1):
        bad = table.clone()
        bad[0, 2], bad[0, 4] = entry, entry
        o, lse = fa.cache_forward_e2m1(q.to(DEV), cache, bad.to(DEV), i32(lens), i32(cu), 0.04, causal=False)
        with pytest.raises(fa.FAError) as e:
            fa.check_errors()
        assert e.value.status == -6 and "site=611" in str(e.value)
        # the same as a request of the remaining keys
        short = torch.tensor([[table[0, j] for j in (0, 1, 3, 5, 6)]], dtype=torch.int32)
        assert_forward(o[:new], lse[:new], q[:new], data, (1., 1.), short, [4 * P + 4], [0, new], 0.04, False)
        assert_forward(o[new:], lse[new:], q[new:], data, (1., 1.), table[1:], lens[1:], [0, new], 0.04, False)
    o, lse = fa.cache_forward_e2m1(q.to(DEV), cache, table.to(DEV), i32([-3, 40]), i32(cu), 0.04)
    with pytest.raises(fa.FAError) as e:
        fa.check_errors()
    assert "site=612" in str(e.value)
    assert (o[:new] == 0).all() and (lse[:new] == -math.inf).all()
    assert_forward(o[new:], lse[new:], q[new:], data, (1., 1.), table[1:], lens[1:], [0, new], 0.04, True)
    o, lse = fa.cache_forward_e2m1(q.to(DEV), cache, table.to(DEV), i32(lens), i32([0, new, 2 * new + 9]), 0.04)
    with pytest.raises(fa.FAError) as e:
        fa.check_errors()
    assert "site=613" in str(e.value)


@pytest.mark.parametrize("P", (16, 64))
@pytest.mark.parametrize("new", (1, 40))
def test_refused_requests_are_not_attended(P, new):
    """With the slot map, a request that cache_slots refused has no keys."""
    R, H, g, d = 3, 1, 4, 64
    table = torch.full((R, 8), -1, dtype=torch.int32)
    table[:, 0] = torch.tensor([0, 1, 2])
    t, lens = table.to(DEV), i32([10, 10, 10])
    n = [new, P + 5, new if new + 10 <= P else 0]
    T = sum(n)
    cu, slots, lens2, used, pos = fa.cache_slots(t, lens, i32(n), i32([3] if P == 64 or new == 1 else [3, 4, 5]), i32([1]
                                                 if P == 64 or new == 1 else [0]), P, T, positions=True)
    data = make_data(8, H, P, d, 2)
    q = _rows(T, H * g, d, 3, -2, 0)
    o, lse = fa.cache_forward_e2m1(q, fa.CacheE2M1(data.to(DEV)), t, lens2, cu, 0.04, slot_map=slots)
    fa.check_errors()
    c, sl, L = cu.tolist(), slots.tolist(), lens2.tolist()
    refused = [r for r in range(R) if c[r + 1] > c[r] and sl[c[r]] < 0]
    assert refused == [1]
    for r in range(R):
        at = slice(c[r], c[r + 1])
        if r in refused:
            assert (o[at] == 0).all() and (lse[at] == -math.inf).all() and (pos[at] == -1).all()
        elif c[r + 1] > c[r]:
            assert pos[at].tolist() == list(range(10, 10 + c[r + 1] - c[r]))
            assert_forward(o[at], lse[at], q[at].cpu(), data, (1., 1.), t[r:r + 1].cpu(), [L[r]],
                           [0, c[r + 1] - c[r]], 0.04, True)


# ------------------------------------------------------------------ a run of them

@pytest.mark.parametrize("P,d,interleaved", ((16, 64, True), (64, 128, False)))
def test_serving_run(P, d, interleaved):
    """Prompts, then single tokens for requests of which some end and one is
    refused for want of blocks: slots and positions, queries turned, appends with
    keys turned on the way, attention."""
    H, g, R, M, units = 2, 2, 4, 8, (2.0 ** -6, 2.0 ** -7)
    blocks = 4 * (-(-70 // P)) - (0 if P == 64 else 3)
    gen = torch.Generator().manual_seed(P)
    free = torch.randperm(blocks, generator=gen).tolist()
    cache = fa.cache_alloc_e2m1(blocks, H, P, d, *units)
    ref = cache.data.cpu().numpy().copy()
    angles = fa.rope_table(200, d // 2)
    table = torch.full((R, M), -1, dtype=torch.int32, device=DEV)
    lens, used = i32([0] * R), i32([0])
    rtable, rlens, rused = table.tolist(), [0] * R, 0
    for step, new in enumerate(([60, 17, 0, 5], [1, 1, 66, 1], [1, 0, 1, 1], [6, 0, 1, 1], [1, 1, 1, 60])):
        T = sum(new) + 3  # three rows of padding
        old = list(rlens)
        cu, slots, lens, used, pos = fa.cache_slots(table, lens, i32(new), i32(free), used, P, T, positions=True)
        rtable, rcu, rslots, rlens, rused = oracle.cache_slots(rtable, rlens, new, free, rused, P, T)
        assert table.tolist() == rtable and slots.tolist() == rslots and lens.tolist() == rlens
        rpos = [-1] * T
        for r in range(R):
            if rlens[r] > old[r]:
                rpos[rcu[r]:rcu[r + 1]] = range(old[r], rlens[r])
        assert pos.tolist() == rpos
        k, v = _rows(T, H, d, 10 + step, -1, 1), _rows(T, H, d, 20 + step, -1, 1)
        q = _rows(T, H * g, d, 30 + step, -2, 1)
        at = np.array(rpos)[:, None]
        turned = fa.rope(q, pos, angles, interleaved=interleaved)
        fa.cache_append_e2m1(k, v, cache, slots, positions=pos, table=angles, interleaved=interleaved)
        o, lse = fa.cache_forward_e2m1(turned, cache, table, lens, cu, slot_map=slots)
        fa.check_errors()
        kr = oracle.rope(k, at, angles, interleaved)
        oracle.cache_e2m1.append(ref, kr.double().numpy(), v.cpu().double().numpy(), rslots, *units)
        _codes_equal(cache.data, ref, f"step {step}")
        want = [0 if rlens[r] == old[r] and new[r] else rlens[r] for r in range(R)]
        assert torch.equal(turned.cpu(), oracle.rope(q, at, angles, interleaved))
        assert_forward(o, lse, turned.cpu(), torch.from_numpy(ref), units, table.cpu(), want, rcu, d ** -0.5, True,
                       f"step {step}")


def test_captured_step_replays_on_new_lengths():
    """A decode step captured once and replayed: the same as calls."""
    P, d, H, g, R = 16, 64, 1, 2, 3
    free, angles = i32(list(range(40))), fa.rope_table(100, d)

    def fresh():
        return (fa.cache_alloc_e2m1(40, H, P, d), torch.full((R, 12), -1, dtype=torch.int32, device=DEV),
                i32([0] * R), i32([0]))

    def step(cache, table, lens, used, k, v, q):
        cu, slots, lens, used, pos = fa.cache_slots(table, lens, one, free, used, P, R, positions=True)
        q = fa.rope(q, pos, angles)
        fa.cache_append_e2m1(k, v, cache, slots, positions=pos, table=angles)
        return fa.cache_forward_e2m1(q, cache, table, lens, cu, slot_map=slots), lens, used

    rows = [(_rows(R, H, d, s, -2, 2), _rows(R, H, d, 50 + s, -2, 2), _rows(R, H * g, d, 90 + s, -1, 1))
            for s in range(20)]
    one = i32([1] * R)
    cache, table, lens, used = fresh()
    want = []
    for k, v, q in rows:
        out, lens, used = step(cache, table, lens, used, k, v, q)
        want.append(out)
    fa.check_errors()
    cache2, table2, lens2, used2 = fresh()
    ks, vs, qs = (t.clone() for t in rows[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        (o, lse), l2, u2 = step(cache2, table2, lens2, used2, ks, vs, qs)
        lens2.copy_(l2)
        used2.copy_(u2)
    for (k, v, q), (ow, lw) in zip(rows, want):
        ks.copy_(k)
        vs.copy_(v)
        qs.copy_(q)
        graph.replay()
        assert torch.equal(o, ow) and torch.equal(lse, lw)
    fa.check_errors()
    assert torch.equal(cache.data, cache2.data)


def test_other_streams():
    lens, P, d = [5000, 10], 16, 64
    table, blocks = make_tables(lens, P, seed=1)
    cache = _cache(blocks, 1, P, d, 2)
    q = _rows(2, 1, d, 1)
    t, sl, cu = table.to(DEV), i32(lens), i32([0, 1, 2])
    want = fa.cache_forward_e2m1(q, cache, t, sl, cu)
    k, v = _rows(3, 1, d, 5), _rows(3, 1, d, 6)
    slots = torch.tensor([1, 9, 4], device=DEV)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for stream in (s, s.cuda_stream):
        got = fa.cache_forward_e2m1(q, cache, t, sl, cu, stream=stream)
        fa.check_errors(s)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    fa.cache_append_e2m1(k, v, cache, slots, stream=s)
    kv = fa.cache_read_e2m1(cache, slots, stream=s)
    fa.check_errors(s)
    assert all(torch.equal(a, b) for a, b in zip(kv, fa.cache_read_e2m1(cache, slots)))


@pytest.mark.parametrize("new", (1, 40))
def test_cache_of_more_than_4_gib(new):
    """Blocks that lie beyond 32-bit offsets: the same bytes and results as in a small cache."""
    H, P, d, g = 8, 128, 128, 4
    blocks = (1 << 32) // (H * P // 16 * 18 * d) + 9
    lens = [150, 300, 40]
    table, few = make_tables(lens, P, seed=new)
    far = torch.where(table >= 0, table + blocks - few, table)
    far[1, 0] = 1  # and one at the start
    T, cu = 3 * new, [0, new, 2 * new, 3 * new]
    k, v = _rows(sum(lens), H, d, 1), _rows(sum(lens), H, d, 2)
    q = _rows(T, H * g, d, 3, -2, 0)
    out = []
    for n, tab in ((few, table), (blocks, far)):
        cache = fa.cache_alloc_e2m1(n, H, P, d)
        slots = torch.tensor([int(tab[r, i // P]) * P + i % P for r, m in enumerate(lens) for i in range(m)], device=DEV)
        fa.cache_append_e2m1(k, v, cache, slots)
        o, lse = fa.cache_forward_e2m1(q, cache, tab.to(DEV), i32(lens), i32(cu))
        used = tab[tab >= 0].long().to(DEV)
        out.append([o, lse, cache.data[used], *fa.cache_read_e2m1(cache, slots)])
    fa.check_errors()
    for a, b in zip(*out):
        assert torch.equal(a, b)


def test_calls_at_once_on_two_streams():
    """Calls that run side by side, each with a workspace of its own."""
    jobs = []
    for i, (lens, new, d) in enumerate((([3000, 900, 50] * 8, 1, 128), ([700, 1200], 150, 64))):
        table, blocks = make_tables(lens, 32, seed=i)
        cu = [new * r for r in range(len(lens) + 1)]
        jobs.append((_rows(cu[-1], 8, d, i, -1, 1), _cache(blocks, 4, 32, d, i), table.to(DEV), i32(lens), i32(cu)))
    want = [fa.cache_forward_e2m1(*job) for job in jobs]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream(), torch.cuda.Stream()], []
    for _ in range(20):
        for job, s, w in zip(jobs, streams, want):
            got.append((fa.cache_forward_e2m1(*job, stream=s), w))
    torch.cuda.synchronize()
    fa.check_errors()
    for (o, lse), (ow, lw) in got:
        assert torch.equal(o, ow) and torch.equal(lse, lw)


def test_captured_prompts_replay_on_other_lengths():
    """Prompts in a graph: tables, lengths and rows of later batches, shorter
    ones and padded ones, as eager calls give them."""
    P, H, g, d, T, R = 64, 2, 4, 128, 200, 3
    batches = [([500, 30, 90], [100, 10, 90]), ([7, 0, 0], [7, 0, 0]), ([640, 600, 64], [64, 72, 64]),
               ([130, 129, 1], [130, 0, 1])]
    gen = torch.Generator().manual_seed(3)
    cache = _cache(40, H, P, d, 1)
    table, lens, cu = i32([[0] * 10] * R), i32([0] * R), i32([0] * (R + 1))
    q = torch.zeros(T, H * g, d, dtype=torch.bfloat16, device=DEV)
    fa.cache_forward_e2m1(q, cache, table, lens, cu)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = fa.cache_forward_e2m1(q, cache, table, lens, cu)
    for n, new in batches:
        table.copy_(torch.randperm(40, generator=gen)[:30].reshape(R, 10).to(torch.int32))
        lens.copy_(i32(n))
        cu.copy_(i32([0, new[0], new[0] + new[1], sum(new)]))
        q.copy_(torch.randn(T, H * g, d, generator=gen).to(torch.bfloat16))
        ow, lw = fa.cache_forward_e2m1(q, cache, table, lens, cu)
        graph.replay()
        rows = sum(new)
        assert torch.equal(o[:rows], ow[:rows]) and torch.equal(lse[:rows], lw[:rows])
    fa.check_errors()


def test_results_are_freed():
    """Call after call takes the same memory."""
    P, d, H, g = 16, 64, 2, 2
    cache = _cache(40, H, P, d, 1)
    q, sl = _rows(3, H * g, d, 2), torch.tensor([1, 2, 3], device=DEV)
    table, lens, cu, angles = i32([[0, 1]] * 3), i32([20, 3, 9]), i32([0, 1, 2, 3]), fa.rope_table(40, d)

    def step():
        fa.cache_append_e2m1(q[:, :H], q[:, H:], cache, sl, positions=lens, table=angles)
        return fa.rope(q, lens, angles), fa.cache_read_e2m1(cache, sl), fa.cache_forward_e2m1(q, cache, table, lens, cu)

    step()
    before = torch.cuda.memory_allocated()
    for _ in range(20):
        step()
    assert torch.cuda.memory_allocated() == before


def test_the_usual_path_and_the_other_agree():
    """The same bits with a stream given (which takes Python's way to the library)
    and without, and a workspace of one's own."""
    P, H, g, d = 32, 2, 4, 128
    lens, new = [300, 70, 5], [20, 1, 5]
    table, blocks = make_tables(lens, P, seed=1)
    cu, T = [0, 20, 21, 26], 26
    qkv, angles = _rows(T, H * (g + 2), d, 3, -1, 1), fa.rope_table(400, 96)
    pos = i32([i for n, a in zip(lens, new) for i in range(n - a, n)])
    sl = torch.tensor([int(table[r, i // P]) * P + i % P for r, (n, a) in enumerate(zip(lens, new))
                       for i in range(n - a, n)], device=DEV)
    outs = []
    for kw in ({}, dict(stream=torch.cuda.current_stream())):
        cache = _cache(blocks, H, P, d, 2)
        q = fa.rope(qkv[:, :H * g], pos, angles, interleaved=True, **kw)
        fa.cache_append_e2m1(qkv[:, H * g:H * (g + 1)], qkv[:, H * (g + 1):], cache, sl, positions=pos, table=angles,
                             interleaved=True, **kw)
        ws = torch.empty(fa.cache_forward_e2m1_workspace_size(3, T, H * g, H, d), dtype=torch.uint8, device=DEV)
        args = (q, cache, table.to(DEV), i32(lens), i32(cu))
        outs.append([q, fa.rope_backward(q, pos, angles, interleaved=True, **kw), cache.data,
                     *fa.cache_read_e2m1(cache, sl, **kw), *fa.cache_forward_e2m1(*args, **kw),
                     *fa.cache_forward_e2m1(*args, slot_map=sl, workspace=ws, causal=False, **kw)])
    fa.check_errors()
    for a, b in zip(*outs):
        assert torch.equal(a, b)
    with pytest.raises(fa.FAError):
        fa.cache_forward_e2m1(*args, workspace=ws[:-8])
    with pytest.raises(fa.FAError):
        fa.cache_read_e2m1(fa.CacheE2M1(cache.data, 3.0, 1.0), sl)
    for bad in (dict(q=q.float()), dict(block_table=args[2].long()), dict(seq_lens=args[3][:2]),
                dict(cu_q=args[4][:3]), dict(slot_map=sl[:3])):
        a = dict(zip(("q", "cache", "block_table", "seq_lens", "cu_q"), args))
        a.update(bad)
        with pytest.raises((TypeError, ValueError)):
            fa.cache_forward_e2m1(**a)


def test_the_same_slot_twice_touches_no_other():
    """Rows of one slot may mix, group by group; every other byte is as it was."""
    P, d, H, T = 32, 128, 2, 8
    k, v = _rows(T, H, d, 1), _rows(T, H, d, 2)
    slots = [5, 5, 5, 9, 9, 40, 5, 63]
    cache = _cache(2, H, P, d, 3)
    ref = cache.data.cpu().numpy().copy()
    fa.cache_append_e2m1(k, v, cache, torch.tensor(slots, device=DEV))
    fa.check_errors()
    got = cache.data.cpu().numpy()
    mine = np.zeros_like(ref, dtype=bool)
    for byte, _, scale in oracle.cache_e2m1.places(d):
        for s in set(slots):
            for where in (byte, scale):
                mine[s // P, :, s % P // 16, where[s % 16]] = True
    assert (got[~mine] == ref[~mine]).all()
    want = ref.copy()
    oracle.cache_e2m1.append(want, k.cpu().double().numpy(), v.cpu().double().numpy(), slots, 1.0, 1.0)
    for s in (40, 63):  # those met once
        once = np.zeros_like(mine)
        for byte, _, scale in oracle.cache_e2m1.places(d):
            for where in (byte, scale):
                once[s // P, :, s % P // 16, where[s % 16]] = True
        a, b = np.where(once, got, 0), np.where(once, want, 0)
        _codes_equal(torch.from_numpy(a), b)
