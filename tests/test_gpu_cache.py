"""The 8-bit key/value cache on the GPU against the float64 oracle: slots and
appended codes exactly, attention within derived bounds
(``cache_cases.forward_bounds``)."""
import math

import numpy as np
import pytest
import torch

import exact_attention_forward_04_gb300 as fa
import oracle
from tests.cache_cases import assert_forward, make_codes, make_tables, poison

pytestmark = pytest.mark.gpu

DEV = "cuda"


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


# ------------------------------------------------------------------- slots

def _slots_case(lens, new, P, F, used, T, M=None, seed=0):
    """cache_slots against the oracle: every output, the table whole."""
    g = torch.Generator().manual_seed(seed)
    held = [-(-max(0, n) // P) for n in lens]
    M = M or max([1] + [-(-(max(0, n) + max(0, a)) // P) for n, a in zip(lens, new)])
    perm = torch.randperm(sum(held) + F, generator=g).tolist()
    table, at = [], 0
    for h in held:
        table.append((perm[at:at + h] + [-7] * M)[:M])
        at += h
    free = perm[at:]
    t = torch.tensor(table, dtype=torch.int32).reshape(len(lens), M).to(DEV)
    out = fa.cache_slots(t, i32(lens), i32(new), i32(free), i32([used]), P, T)
    fa.check_errors()
    ref = oracle.cache_slots(table, lens, new, free, used, P, T)
    got = (t.tolist(), out[0].tolist(), out[1].tolist(), out[2].tolist(), out[3].item())
    for name, a, b in zip(("table", "cu", "slots", "lens", "used"), got, ref):
        assert a == b, name
    assert [x.dtype for x in out] == [torch.int32, torch.int64, torch.int32, torch.int32]


@pytest.mark.parametrize("P", (16, 32, 64, 128))
@pytest.mark.parametrize("R,high", ((1, 1), (3, 200), (37, 500), (1500, 3)))
def test_slots_ragged(P, R, high):
    g = torch.Generator().manual_seed(R + P)
    lens = torch.randint(0, 400, (R,), generator=g).tolist()
    new = torch.randint(0, high + 1, (R,), generator=g).tolist()
    _slots_case(lens, new, P, F=sum(-(-n // P) for n in new) + R + 4, used=3, T=sum(new) + 9, seed=R)


@pytest.mark.parametrize("F", (0, 1, 5, 6, 40))
def test_slots_free_blocks_run_out(F):
    # a prefix of the requests that need blocks is served, and those that need none
    _slots_case([0, 16, 15, 3, 32, 7, 1], [40, 1, 1, 13, 20, 2, 100], 16, F=F, used=0, T=300)


def test_slots_used_beyond_the_list_and_short_map_and_table():
    _slots_case([0, 5, 16], [3, 2, 1], 16, F=4, used=9, T=20)
    _slots_case([0, 5, 16, 2], [3, 20, 1, 1], 16, F=4, used=0, T=10)    # the second and later ones exceed the map
    _slots_case([0, 5, 16, 2], [3, 40, 1, 1], 16, F=4, used=0, T=100, M=2)  # the second exceeds its table row
    _slots_case([-4, 5], [-3, 2], 16, F=2, used=0, T=4)                 # negative lengths count as 0


def test_slots_without_requests_or_tokens():
    _slots_case([], [], 32, F=2, used=1, T=5, M=1)
    _slots_case([4, 9], [0, 0], 32, F=0, used=0, T=0)


def test_slots_more_requests_than_threads():
    g = torch.Generator().manual_seed(5)
    R = 2500
    lens = torch.randint(0, 70, (R,), generator=g).tolist()
    new = torch.randint(0, 4, (R,), generator=g).tolist()
    _slots_case(lens, new, 16, F=R, used=0, T=sum(new))


# ------------------------------------------------------------------ append

def _append_ref(k, v, cache, slots, P):
    out = [t.cpu().numpy().copy() for t in cache]
    oracle.cache_append(k.float().cpu().numpy(), out[0], out[2], slots, P)
    oracle.cache_append(v.float().cpu().numpy(), out[1], out[3], slots, P)
    return out


def _same(cache, ref, what=""):
    for name, a, b in zip(cache._fields, cache, ref):
        assert np.array_equal(a.cpu().numpy(), b), f"{what}: {name}"


def _random_cache(blocks, H, P, d, seed):
    k8, ks = make_codes(blocks, H, P, d, seed)
    v8, vs = make_codes(blocks, H, P, d, seed + 1)
    return fa.CacheE4M3(*(t.to(DEV) for t in (k8, v8, ks, vs)))


def _rows(T, H, d, seed, low=-6, high=6):
    """bf16 rows of magnitudes 2^low .. 2^high, and a few zeros."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, H, d, generator=g) * torch.exp2(torch.randint(low, high + 1, (T, H, 1), generator=g).float())
    return x.to(torch.bfloat16).to(DEV)


@pytest.mark.parametrize("P", (16, 32, 64, 128))
@pytest.mark.parametrize("d", (64, 128))
@pytest.mark.parametrize("H", (1, 3))
def test_append_prompts(P, d, H):
    """Ragged runs: new blocks, starts inside blocks, a block's last slot, runs of one."""
    held, new = [0, 5, P - 1, 2 * P, 3, 0], [P + 3, 1, 2, 2 * P, 3 * P, 1]
    table, blocks = make_tables([h + n for h, n in zip(held, new)], P, seed=P)
    slots = [int(table[r, p // P]) * P + p % P for r in range(6) for p in range(held[r], held[r] + new[r])]
    cache = _random_cache(blocks, H, P, d, seed=P + d)
    k, v = _rows(len(slots), H, d, 1), _rows(len(slots), H, d, 2)
    ref = _append_ref(k, v, cache, slots, P)
    fa.cache_append_e4m3(k, v, cache, torch.tensor(slots, device=DEV))
    fa.check_errors()
    _same(cache, ref, f"P={P} d={d}")


@pytest.mark.parametrize("T,H", ((300, 3), (900, 5), (2500, 8), (2500, 19), (9000, 9)))
@pytest.mark.parametrize("P,d", ((16, 64), (64, 128), (128, 128)))
def test_append_many_tokens(T, H, P, d):
    """Runs of one token among longer ones, over all the shares of a call that
    a CTA takes: few tokens of one head to many of several, K's and V's."""
    gen = torch.Generator().manual_seed(T + P)
    slots, block = [], 0
    while len(slots) < T:
        kind = int(torch.randint(0, 4, (1,), generator=gen))
        if kind == 3:
            slots.append(-1)
            continue
        n = 1 if kind == 0 else int(torch.randint(2, 3 * P, (1,), generator=gen))
        at = block * P + int(torch.randint(0, P, (1,), generator=gen))
        slots += range(at, at + n)
        block = (at + n + P - 1) // P + 1  # no block is met twice
    slots = slots[:T]
    cache = _random_cache(block, H, P, d, seed=T)
    k, v = _rows(T, H, d, 1), _rows(T, H, d, 2)
    ref = _append_ref(k, v, cache, slots, P)
    fa.cache_append_e4m3(k, v, cache, torch.tensor(slots, device=DEV))
    fa.check_errors()
    _same(cache, ref, f"T={T} H={H} P={P} d={d}")


@pytest.mark.parametrize("P,d", ((16, 128), (128, 64)))
def test_append_token_by_token(P, d):
    """Two blocks filled one token at a time, magnitudes rising and falling."""
    cache = fa.cache_alloc_e4m3(4, 2, P, d)
    n = P + 5
    k, v = _rows(n, 2, d, 3, -12, 12), _rows(n, 2, d, 4, -12, 12)
    k[3] = 0
    blocks = [2, 0]
    ref = [t.cpu().numpy() for t in cache]
    for i in range(n):
        slot = [blocks[i // P] * P + i % P]
        oracle.cache_append(k[i:i + 1].float().cpu().numpy(), ref[0], ref[2], slot, P)
        oracle.cache_append(v[i:i + 1].float().cpu().numpy(), ref[1], ref[3], slot, P)
        fa.cache_append_e4m3(k[i:i + 1], v[i:i + 1], cache, torch.tensor(slot, device=DEV))
    fa.check_errors()
    _same(cache, ref)


def test_append_extreme_magnitudes():
    """Zeros, the smallest and largest bf16, values whose scale meets its limits, ties."""
    P, d = 16, 64
    vals = [0.0, 2.0 ** -133, -2.0 ** -126, 2.0 ** -92, 448 * 2.0 ** -100, 449 * 2.0 ** -100, 1.75, 1.7578125, 240.0,
            448.0, 450.0, 3.3895313892515355e38, -3.3895313892515355e38, 17.0, 19.0]
    cache = fa.cache_alloc_e4m3(len(vals), 1, P, d)
    k = torch.zeros(len(vals), 1, d)
    for i, x in enumerate(vals):
        k[i, 0, 3], k[i, 0, 5], k[i, 0, 63] = x, x / 16, -x / 4096
    k = k.to(torch.bfloat16).to(DEV)
    slots = [i * P for i in range(len(vals))]
    ref = _append_ref(k, -k, cache, slots, P)
    fa.cache_append_e4m3(k, -k, cache, torch.tensor(slots, device=DEV))
    fa.check_errors()
    _same(cache, ref)


def test_append_strided_rows_and_skipped_slots():
    """K and V as slices of one projection; -1 slots inside a run end it."""
    P, d, H = 32, 128, 2
    T = 50
    qkv = _rows(T, 7 * H, d, 9)
    k, v = qkv[:, 3 * H:4 * H], qkv[:, 5 * H:6 * H]
    slots = list(range(40, 40 + T))
    for i in (0, 7, 8, 49):
        slots[i] = -1
    slots[30] = 5  # a block of its own
    cache = _random_cache(4, H, P, d, 11)
    ref = _append_ref(k, v, cache, slots, P)
    # rows 9..23 and 31.. start inside blocks that rows before them wrote to:
    # two runs of one block in a call are not allowed, so append them apart
    for part in (range(0, 8), range(8, 31), range(31, T)):
        some = [slots[i] if i in part else -1 for i in range(T)]
        fa.cache_append_e4m3(k, v, cache, torch.tensor(some, device=DEV))
    fa.check_errors()
    _same(cache, ref)


def test_append_reports_slots_out_of_range():
    P, d, H = 16, 64, 1
    cache = _random_cache(3, H, P, d, 12)
    k, v = _rows(4, H, d, 5), _rows(4, H, d, 6)
    slots = [3, 48, -2, 1 << 40]
    ref = _append_ref(k, v, cache, slots, P)
    fa.cache_append_e4m3(k, v, cache, torch.tensor(slots, device=DEV))
    with pytest.raises(fa.FAError) as e:
        fa.check_errors()
    assert e.value.status == -6 and "site=601" in str(e.value)
    fa.check_errors()  # reported once
    _same(cache, ref)


def test_append_nothing():
    cache = _random_cache(2, 1, 16, 64, 13)
    before = [t.clone() for t in cache]
    fa.cache_append_e4m3(_rows(0, 1, 64, 1), _rows(0, 1, 64, 1), cache, torch.empty(0, dtype=torch.int64, device=DEV))
    fa.check_errors()
    assert all(torch.equal(a, b) for a, b in zip(cache, before))


# ----------------------------------------------------------------- forward

def _forward_case(lens, new, P, H, g, d, causal=True, scale=None, seed=0, sigma=1.0, **kw):
    table, blocks = make_tables(lens, P, seed=seed)
    k8, ks = make_codes(blocks, H, P, d, seed + 1)
    v8, vs = make_codes(blocks, H, P, d, seed + 2)
    poison(k8, table, lens)
    poison(v8, table, lens)
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    gen = torch.Generator().manual_seed(seed + 3)
    q = (torch.randn(cu[-1] + 2, H * g, d, generator=gen) * sigma).to(torch.bfloat16)  # two rows of no request
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    cache = fa.CacheE4M3(*(t.to(DEV) for t in (k8, v8, ks, vs)))
    o, lse = fa.cache_forward_e4m3(q.to(DEV), cache, table.to(DEV), i32(lens), i32(cu), scale=scale, causal=causal,
                                   **kw)
    fa.check_errors()
    what = f"lens={lens[:4]} new={new[:4]} P={P} H={H} g={g} d={d} causal={causal}"
    return assert_forward(o, lse, q, (k8, v8, ks, vs), table, lens, cu, scale, causal, what)


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
def test_forward_prompts_not_causal_and_negative_scale(d):
    _forward_case([200, 90], [70, 90], 32, 2, 4, d, causal=False, seed=3)
    _forward_case([200, 90], [70, 90], 64, 1, 4, d, scale=-0.15, seed=4)
    _forward_case([200, 90], [70, 90], 16, 1, 4, d, scale=0.0, seed=5)


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


@pytest.mark.parametrize("d", (64, 128))
@pytest.mark.parametrize("g,high", ((1, 1), (4, 2), (12, 2), (12, 30)))
def test_forward_many_pieces_the_same_every_time(d, g, high):
    """Many units of very different lengths a CTA, so that short pieces run
    side by side while longer ones wait for their keys: the same bits from
    every call, and right."""
    gen = torch.Generator().manual_seed(g + d)
    R, H, P = 160, 8, 16
    lens = (torch.randint(0, 40, (R,), generator=gen) ** 2).tolist()
    new = [min(n, int(x)) for n, x in zip(lens, torch.randint(0, high + 1, (R,), generator=gen))]
    table, blocks = make_tables(lens, P, seed=g)
    codes = make_codes(blocks, H, P, d, 1) + make_codes(blocks, H, P, d, 2)
    k8, ks, v8, vs = codes
    poison(k8, table, lens)
    poison(v8, table, lens)
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    q = torch.randn(cu[-1], H * g, d, generator=gen).to(torch.bfloat16)
    args = (q.to(DEV), fa.CacheE4M3(*(t.to(DEV) for t in (k8, v8, ks, vs))), table.to(DEV), i32(lens), i32(cu))
    o, lse = fa.cache_forward_e4m3(*args)
    for _ in range(40):
        o2, lse2 = fa.cache_forward_e4m3(*args)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
    fa.check_errors()
    h = 5  # one kv head of the whole batch against the oracle
    at, of = slice(h * g, h * g + g), slice(h, h + 1)
    assert_forward(o[:, at], lse[:, at], q[:, at], (k8[:, of], v8[:, of], ks[:, of], vs[:, of]), table, lens, cu,
                   d ** -0.5, True, f"d={d} g={g}")


def test_forward_wide_groups_and_heads():
    _forward_case([130, 50], [1, 1], 64, 1, 40, 128, seed=5)   # more rows than a tile
    _forward_case([70], [1], 32, 24, 1, 64, seed=6)


@pytest.mark.parametrize("scale", (0.0, -0.1, 2.0))
def test_forward_scales(scale):
    _forward_case([100, 33], [1, 2], 32, 1, 2, 64, scale=scale, seed=7)


def test_forward_peaky_rows():
    _forward_case([500, 260], [1, 4], 64, 2, 4, 128, sigma=8.0, seed=8)


@pytest.mark.parametrize("d", (64, 128))
@pytest.mark.parametrize("rows", (1, 20))
def test_forward_blocks_of_very_different_scale(d, rows):
    """V blocks of zeros with the smallest scale beside large ones; the
    weights of small blocks stay exact where the large ones' vanish."""
    P, lens = 16, [96, 64]
    table, blocks = make_tables(lens, P, seed=1)
    k8, ks = make_codes(blocks, 1, P, d, 2)
    v8, vs = make_codes(blocks, 1, P, d, 3)
    v8[table[0, 0].item()] = 0
    vs[table[0, 0].item()] = 2.0 ** -100
    v8[table[1, 2].item()] = 0                # and one whose keys are seen
    vs[table[1, 2].item()] = 2.0 ** -100
    vs[table[0, 3].item()] = 2.0 ** 40
    k8[table[0, 3].item()] = k8[table[0, 3].item()] | 0x80  # its scores are far below the others'
    cu = [0, rows, 2 * rows]
    q = torch.full((2 * rows, 2, d), 1.0, dtype=torch.bfloat16)
    k8[table[0, 1].item()] &= 0x7F
    ks[table[0, 1].item()] = 1.0
    ks[table[0, 3].item()] = 4.0
    cache = fa.CacheE4M3(*(t.to(DEV) for t in (k8, v8, ks, vs)))
    o, lse = fa.cache_forward_e4m3(q.to(DEV), cache, table.to(DEV), i32(lens), i32(cu))
    fa.check_errors()
    assert_forward(o, lse, q, (k8, v8, ks, vs), table, lens, cu, 1 / math.sqrt(d), True)


@pytest.mark.parametrize("g", (2, 34))
def test_forward_query_magnitudes(g):
    """Rows of any magnitude, zeros, and elements far below a row's largest."""
    lens, P, d = [60, 60, 60, 60], 32, 64
    table, blocks = make_tables(lens, P, seed=1)
    k8, ks = make_codes(blocks, 1, P, d, 2)
    v8, vs = make_codes(blocks, 1, P, d, 3)
    q = torch.randn(4, g, d, generator=torch.Generator().manual_seed(4))
    q[0] *= 2.0 ** -130
    q[1] = 0
    q[2] *= torch.exp2(-torch.arange(d).float())
    q[3, 1] *= 2.0 ** 100
    scales = 1.0
    q = q.to(torch.bfloat16)
    cache = fa.CacheE4M3(*(t.to(DEV) for t in (k8, v8, ks, vs)))
    o, lse = fa.cache_forward_e4m3(q.to(DEV), cache, table.to(DEV), i32(lens), i32([0, 1, 2, 3, 4]), scale=scales)
    fa.check_errors()
    # the row of 2^100 has scores beyond 2^100: one key takes all the weight
    assert_forward(o, lse, q, (k8, v8, ks, vs), table, lens, [0, 1, 2, 3, 4], scales, True)


@pytest.mark.parametrize("d", (64, 128))
@pytest.mark.parametrize("g", (2, 5, 12, 34))
def test_forward_rows_that_are_not_finite(d, g):
    """A query row of NaNs and one of infinities leave the others as they are."""
    lens, P = [100, 300], 32
    table, blocks = make_tables(lens, P, seed=1)
    k8, ks = make_codes(blocks, 1, P, d, 2)
    v8, vs = make_codes(blocks, 1, P, d, 3)
    cache = fa.CacheE4M3(*(t.to(DEV) for t in (k8, v8, ks, vs)))
    q = torch.randn(2, g, d, generator=torch.Generator().manual_seed(g)).to(torch.bfloat16)
    bad = q.clone()
    bad[0, 0], bad[1, 1] = math.nan, math.inf
    o, lse = fa.cache_forward_e4m3(bad.to(DEV), cache, table.to(DEV), i32(lens), i32([0, 1, 2]))
    fa.check_errors()
    keep = [[h for h in range(g) if h != r] for r in (0, 1)]
    for r in (0, 1):
        assert_forward(o[r:r + 1, keep[r]], lse[r:r + 1, keep[r]], q[r:r + 1, keep[r]], (k8, v8, ks, vs),
                       table[r:r + 1], lens[r:r + 1], [0, 1], d ** -0.5, True, f"row {r}")


def test_forward_strided_queries_untouched_rows_and_repeatability():
    lens, new, P, d = [200, 31, 0], [2, 1, 0], 32, 128
    table, blocks = make_tables(lens, P, seed=1)
    k8, ks = make_codes(blocks, 2, P, d, 2)
    v8, vs = make_codes(blocks, 2, P, d, 3)
    cache = fa.CacheE4M3(*(t.to(DEV) for t in (k8, v8, ks, vs)))
    big = torch.randn(6, 12, d, generator=torch.Generator().manual_seed(4)).to(torch.bfloat16).to(DEV)
    q = big[:, 2:6]
    ws = torch.full((fa.cache_forward_workspace_size(3, 6, 4, 2, d),), 0xFF, dtype=torch.uint8, device=DEV)
    o, lse = fa.cache_forward_e4m3(q, cache, table.to(DEV), i32(lens), i32([0, 2, 3, 3]), workspace=ws)
    assert_forward(o[:3], lse[:3], q[:3].cpu(), (k8, v8, ks, vs), table, lens, [0, 2, 3, 3], d ** -0.5, True)
    lib = fa.load_library()
    o2, lse2 = torch.full_like(o, 7.0), torch.full_like(lse, 7.0)
    t, sl, cu = table.to(DEV), i32(lens), i32([0, 2, 3, 3])
    st = lib.fa_cache_fwd_e4m3(q.data_ptr(), q.stride(0), *(c.data_ptr() for c in cache), t.data_ptr(), sl.data_ptr(),
                               cu.data_ptr(), o2.data_ptr(), lse2.data_ptr(), 3, 6, 4, 2, d, blocks, P, t.shape[1],
                               d ** -0.5, 1, ws.data_ptr(), ws.numel(), torch.cuda.current_stream().cuda_stream)
    assert st == 0
    fa.check_errors()
    assert torch.equal(o2[:3], o[:3]) and torch.equal(lse2[:3], lse[:3])
    assert (o2[3:] == 7).all() and (lse2[3:] == 7).all()


def test_forward_reports_what_is_out_of_range():
    """Blocks outside the cache hide their keys; lengths and rows are cut off."""
    lens, P, d = [100, 40], 16, 64
    table, blocks = make_tables(lens, P, seed=1)
    k8, ks = make_codes(blocks, 1, P, d, 2)
    v8, vs = make_codes(blocks, 1, P, d, 3)
    q = torch.randn(2, 1, d, generator=torch.Generator().manual_seed(4)).to(torch.bfloat16)
    cache = fa.CacheE4M3(*(t.to(DEV) for t in (k8, v8, ks, vs)))
    bad = table.clone()
    bad[0, 2], bad[0, 6] = blocks, -5
    o, lse = fa.cache_forward_e4m3(q.to(DEV), cache, bad.to(DEV), i32(lens), i32([0, 1, 2]))
    with pytest.raises(fa.FAError) as e:
        fa.check_errors()
    assert e.value.status == -6 and "site=611" in str(e.value)
    # the same as a request of the remaining keys
    short = torch.tensor([[table[0, j] for j in (0, 1, 3, 4, 5)]], dtype=torch.int32)
    assert_forward(o[:1], lse[:1], q[:1], (k8, v8, ks, vs), short, [80], [0, 1], d ** -0.5, True)
    assert_forward(o[1:], lse[1:], q[1:], (k8, v8, ks, vs), table[1:], lens[1:], [0, 1], d ** -0.5, True)
    M = table.shape[1]
    o, lse = fa.cache_forward_e4m3(q.to(DEV), cache, table.to(DEV), i32([-3, 40]), i32([0, 1, 2]))
    with pytest.raises(fa.FAError) as e:
        fa.check_errors()
    assert "site=612" in str(e.value)
    assert (o[0] == 0).all() and (lse[0] == -math.inf).all()
    assert_forward(o[1:], lse[1:], q[1:], (k8, v8, ks, vs), table[1:], lens[1:], [0, 1], d ** -0.5, True)
    full, fblocks = make_tables([M * P], P, extra_cols=0, seed=2)
    o, lse = fa.cache_forward_e4m3(q[:1].to(DEV), cache, full.clamp(max=blocks - 1).to(DEV), i32([M * P + 5]),
                                   i32([0, 9]))
    with pytest.raises(fa.FAError) as e:
        fa.check_errors()
    assert "site=61" in str(e.value)
    assert_forward(o, lse, q[:1], (k8, v8, ks, vs), full.clamp(max=blocks - 1), [M * P], [0, 1], d ** -0.5, True)


# ------------------------------------------------------------------ a run of them

@pytest.mark.parametrize("P,d", ((16, 64), (64, 128)))
def test_serving_run(P, d):
    """Prompts, then single tokens for requests of which some end and one is
    refused for want of blocks: slots, appends and attention together."""
    H, g, R, M = 2, 2, 4, 8
    blocks = 4 * (-(-70 // P)) - (0 if P == 64 else 3)
    gen = torch.Generator().manual_seed(P)
    free = torch.randperm(blocks, generator=gen).tolist()
    cache = fa.cache_alloc_e4m3(blocks, H, P, d)
    ref = [t.cpu().numpy() for t in cache]
    table = torch.full((R, M), -1, dtype=torch.int32, device=DEV)
    lens, used = i32([0] * R), i32([0])
    rtable, rlens, rused = table.tolist(), [0] * R, 0
    for step, new in enumerate(([60, 17, 0, 5], [1, 1, 66, 1], [1, 0, 1, 1], [6, 0, 1, 1], [1, 1, 1, 60])):
        T = sum(new) + 3  # three rows of padding
        cu, slots, lens, used = fa.cache_slots(table, lens, i32(new), i32(free), used, P, T)
        rtable, rcu, rslots, rlens, rused = oracle.cache_slots(rtable, rlens, new, free, rused, P, T)
        assert table.tolist() == rtable and slots.tolist() == rslots and lens.tolist() == rlens
        k, v = _rows(T, H, d, 10 + step, -3, 3), _rows(T, H, d, 20 + step, -3, 3)
        q = _rows(T, H * g, d, 30 + step, -2, 1)
        fa.cache_append_e4m3(k, v, cache, slots)
        oracle.cache_append(k.float().cpu().numpy(), ref[0], ref[2], rslots, P)
        oracle.cache_append(v.float().cpu().numpy(), ref[1], ref[3], rslots, P)
        o, lse = fa.cache_forward_e4m3(q, cache, table, lens, cu)
        fa.check_errors()
        _same(cache, ref, f"step {step}")
        assert_forward(o, lse, q.cpu(), [torch.from_numpy(a) for a in ref], table.cpu(), rlens, rcu, d ** -0.5, True,
                       f"step {step}")


def test_captured_step_replays_on_new_lengths():
    """A decode step captured once and replayed: the same as calls."""
    P, d, H, g, R = 16, 64, 1, 2, 3
    free = i32(list(range(40)))

    def fresh():
        return (fa.cache_alloc_e4m3(40, H, P, d), torch.full((R, 12), -1, dtype=torch.int32, device=DEV),
                i32([0] * R), i32([0]))

    rows = [(_rows(R, H, d, s, -2, 2), _rows(R, H, d, 50 + s, -2, 2), _rows(R, H * g, d, 90 + s, -1, 1))
            for s in range(20)]
    one = i32([1] * R)
    cache, table, lens, used = fresh()
    want = []
    for k, v, q in rows:
        cu, slots, lens, used = fa.cache_slots(table, lens, one, free, used, P, R)
        fa.cache_append_e4m3(k, v, cache, slots)
        want.append(fa.cache_forward_e4m3(q, cache, table, lens, cu))
    fa.check_errors()
    cache2, table2, lens2, used2 = fresh()
    ks, vs, qs = (t.clone() for t in rows[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cu, slots, l2, u2 = fa.cache_slots(table2, lens2, one, free, used2, P, R)
        fa.cache_append_e4m3(ks, vs, cache2, slots)
        o, lse = fa.cache_forward_e4m3(qs, cache2, table2, l2, cu)
        lens2.copy_(l2)
        used2.copy_(u2)
    for (k, v, q), (ow, lw) in zip(rows, want):
        ks.copy_(k)
        vs.copy_(v)
        qs.copy_(q)
        graph.replay()
        assert torch.equal(o, ow) and torch.equal(lse, lw)
    fa.check_errors()
    assert all(torch.equal(a, b) for a, b in zip(cache, cache2))


def test_other_streams():
    """A given stream, by object and by handle, carries the whole call."""
    lens, P, d = [5000, 10], 16, 64
    table, blocks = make_tables(lens, P, seed=1)
    k8, ks = make_codes(blocks, 1, P, d, 2)
    v8, vs = make_codes(blocks, 1, P, d, 3)
    cache = fa.CacheE4M3(*(t.to(DEV) for t in (k8, v8, ks, vs)))
    q = _rows(2, 1, d, 1)
    t, sl, cu = table.to(DEV), i32(lens), i32([0, 1, 2])
    want = fa.cache_forward_e4m3(q, cache, t, sl, cu)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for stream in (s, s.cuda_stream):
        got = fa.cache_forward_e4m3(q, cache, t, sl, cu, stream=stream)
        fa.check_errors(s)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("new", (1, 40))
def test_cache_of_more_than_4_gib(new):
    """Blocks whose codes lie beyond 32-bit offsets: the same codes, scales and
    results as in a small cache, with both kernels of the forward."""
    H, P, d, g = 8, 128, 128, 4
    blocks = (1 << 32) // (H * P * d) + 9
    lens = [150, 300, 40]
    table, few = make_tables(lens, P, seed=new)
    far = torch.where(table >= 0, table + blocks - few, table)
    far[1, 0] = 1  # and one at the start
    T, cu = 3 * new, [0, new, 2 * new, 3 * new]
    k, v = _rows(sum(lens), H, d, 1), _rows(sum(lens), H, d, 2)
    q = _rows(T, H * g, d, 3, -2, 0)
    out = []
    for n, tab in ((few, table), (blocks, far)):
        cache = fa.cache_alloc_e4m3(n, H, P, d)
        slots = [int(tab[r, i // P]) * P + i % P for r, m in enumerate(lens) for i in range(m)]
        fa.cache_append_e4m3(k, v, cache, torch.tensor(slots, device=DEV))
        o, lse = fa.cache_forward_e4m3(q, cache, tab.to(DEV), i32(lens), i32(cu))
        used = tab[tab >= 0].long().to(DEV)
        out.append([o, lse] + [t[used] for t in cache])
    fa.check_errors()
    for a, b in zip(*out):
        assert torch.equal(a, b)


def test_calls_at_once_on_two_streams():
    """Calls that run side by side, each with a workspace of its own."""
    jobs = []
    for i, (lens, new, d) in enumerate((([3000, 900, 50] * 8, 1, 128), ([700, 1200], 150, 64))):
        table, blocks = make_tables(lens, 32, seed=i)
        codes = make_codes(blocks, 4, 32, d, i) + make_codes(blocks, 4, 32, d, 9 + i)
        cache = fa.CacheE4M3(*(codes[j].to(DEV) for j in (0, 2, 1, 3)))
        cu = [new * r for r in range(len(lens) + 1)]
        jobs.append((_rows(cu[-1], 8, d, i, -1, 1), cache, table.to(DEV), i32(lens), i32(cu)))
    want = [fa.cache_forward_e4m3(*job) for job in jobs]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream(), torch.cuda.Stream()], []
    for _ in range(20):
        for job, s, w in zip(jobs, streams, want):
            got.append((fa.cache_forward_e4m3(*job, stream=s), w))
    torch.cuda.synchronize()
    fa.check_errors()
    for (o, lse), (ow, lw) in got:
        assert torch.equal(o, ow) and torch.equal(lse, lw)


@pytest.mark.parametrize("d,rows", ((64, 3), (64, 50), (128, 3), (128, 50)))
def test_queries_as_a_slice_of_a_projection(d, rows):
    """Queries, keys and values of one tensor, as strided slices; the same as copies."""
    lens, P, H, g = [rows, rows, rows], 32, 2, 4
    table, blocks = make_tables(lens, P, seed=d)
    qkv = _rows(3 * rows, H * (g + 2) + 1, d, rows, -1, 1)
    q, k, v = qkv[:, :H * g], qkv[:, H * g:H * (g + 1)], qkv[:, H * (g + 1):-1]
    slots = torch.tensor([int(table[r, i // P]) * P + i % P for r in range(3) for i in range(rows)], device=DEV)
    cu, out = i32([0, rows, 2 * rows, 3 * rows]), []
    for x, y, z in ((q, k, v), (q.contiguous(), k.contiguous(), v.contiguous())):
        cache = fa.cache_alloc_e4m3(blocks, H, P, d)
        fa.cache_append_e4m3(y, z, cache, slots)
        out.append((*cache, *fa.cache_forward_e4m3(x, cache, table.to(DEV), i32(lens), cu)))
    fa.check_errors()
    for a, b in zip(*out):
        assert torch.equal(a, b)
    codes = [t.cpu() for t in out[0][:4]]
    assert_forward(out[0][4], out[0][5], q.cpu().contiguous(), codes, table, lens, [0, rows, 2 * rows, 3 * rows],
                   d ** -0.5, True)


def test_captured_prompts_replay_on_other_lengths():
    """The many-row kernel in a graph: tables, lengths and rows of later batches,
    shorter ones and padded ones, as eager calls give them."""
    P, H, g, d, T, R = 64, 2, 4, 128, 200, 3
    batches = [([500, 30, 90], [100, 10, 90]), ([7, 0, 0], [7, 0, 0]), ([640, 600, 64], [64, 72, 64]),
               ([130, 129, 1], [130, 0, 1])]
    gen = torch.Generator().manual_seed(3)
    cache = fa.CacheE4M3(*(t.to(DEV) for t in (make_codes(40, H, P, d, 1)[0], make_codes(40, H, P, d, 2)[0],
                                               make_codes(40, H, P, d, 1)[1], make_codes(40, H, P, d, 2)[1])))
    table, lens, cu = i32([[0] * 10] * R), i32([0] * R), i32([0] * (R + 1))
    q = torch.zeros(T, H * g, d, dtype=torch.bfloat16, device=DEV)
    fa.cache_forward_e4m3(q, cache, table, lens, cu)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = fa.cache_forward_e4m3(q, cache, table, lens, cu)
    for n, new in batches:
        table.copy_(torch.randperm(40, generator=gen)[:30].reshape(R, 10).to(torch.int32))
        lens.copy_(i32(n))
        cu.copy_(i32([0, new[0], new[0] + new[1], sum(new)]))
        q.copy_(torch.randn(T, H * g, d, generator=gen).to(torch.bfloat16))
        ow, lw = fa.cache_forward_e4m3(q, cache, table, lens, cu)
        graph.replay()
        rows = sum(new)
        assert torch.equal(o[:rows], ow[:rows]) and torch.equal(lse[:rows], lw[:rows])
    fa.check_errors()
