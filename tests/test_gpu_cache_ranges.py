"""The 8-bit cache's forward at the ends of its ranges, with the kernel that
each case takes asserted: query rows, scales and scores of any magnitude, V
scales far apart, what is out of range, and batches of every kind for the
many-row kernel.  Against the float64 oracle, within
``cache_cases.forward_bounds`` where nothing else is said."""
import math

import pytest
import torch

import exact_attention_forward_04_gb300 as fa
import oracle
from tests.cache_cases import assert_forward, make_codes, make_tables, poison

pytestmark = pytest.mark.gpu

DEV = "cuda"

# (query heads per kv head, new tokens of a request) of one request on one kv
# head, for the three forms: 8 rows a unit, 16, and the many-row kernel
FORMS = {"few8": (2, 3), "few16": (5, 3), "many": (17, 3)}


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def assert_takes(form, R, T, Hq, H, d):
    """The form follows from the partials' size: two of a unit's rows per CTA."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    rows = {"few8": 8, "few16": 16, "many": 256}[form]
    ctas = sms * (2 if form == "few8" and d == 64 else 1)
    assert fa.cache_forward_workspace_size(R, T, Hq, H, d) == 32 * ctas + 16 + 2 * ctas * rows * (d + 1) * 4


def attend(form, q, codes, table, lens, new, scale=None, causal=True, raises=None, **kw):
    """(o, lse) of the kernel that ``form`` names, cu; ``raises``: the site it reports."""
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    T, Hq, d = q.shape
    assert_takes(form, len(lens), T, Hq, codes[0].shape[1], d)
    cache = fa.CacheE4M3(*(t.to(DEV) for t in codes))
    o, lse = fa.cache_forward_e4m3(q.to(DEV), cache, table.to(DEV), i32(lens), i32(cu), scale=scale, causal=causal,
                                   **kw)
    if raises is None:
        fa.check_errors()
    else:
        with pytest.raises(fa.FAError) as e:
            fa.check_errors()
        assert e.value.status == -6 and f"site={raises}" in str(e.value)
    return o, lse, cu


def check(form, q, codes, table, lens, new, scale, causal=True, what=""):
    o, lse, cu = attend(form, q, codes, table, lens, new, scale, causal)
    return assert_forward(o, lse, q, codes, table, lens, cu, scale, causal, f"{form} {what}")


def one_head(blocks, P, d, seed, k_exp=0, v_exp=0):
    """Random codes of one kv head, scales 2^k_exp and 2^v_exp."""
    k8, ks = make_codes(blocks, 1, P, d, seed, k_exp + 4, k_exp + 4)
    v8, vs = make_codes(blocks, 1, P, d, seed + 1, v_exp + 4, v_exp + 4)
    return k8, v8, ks, vs


# ------------------------------------------------- query rows of any magnitude

@pytest.mark.parametrize("m", (127, 126, 123, 122, 121, -118, -119, -120, -123, -126, -130))
@pytest.mark.parametrize("d", (64, 128))
@pytest.mark.parametrize("form", FORMS)
def test_query_rows_of_any_magnitude(form, d, m):
    """Rows whose largest element lies in [2^m, 2^(m+1)), m the largest of bf16
    and below the smallest normal one, beside keys and a scale that bring the
    scores to a few units; and a row of zeros."""
    g, n = FORMS[form]
    lens, P = [70], 32
    table, blocks = make_tables(lens, P, seed=1)
    k_exp = -98 if m > 0 else 112
    codes = one_head(blocks, P, d, 2, k_exp)
    q = torch.randn(n, g, d, generator=torch.Generator().manual_seed(4), dtype=torch.float64)
    q = q / q.abs().amax(-1, keepdim=True) * 1.5 * 2.0 ** m
    q[1, 0] = 0
    check(form, q.to(torch.bfloat16), codes, table, lens, [n], 2.0 ** -(m + k_exp + 6), what=f"m={m}")


@pytest.mark.parametrize("form", FORMS)
def test_a_scale_of_zero_beside_the_largest_keys(form):
    """Scores of 0 whatever the keys are: the mean of the visible values."""
    g, n = FORMS[form]
    lens, P, d = [70], 32, 64
    table, blocks = make_tables(lens, P, seed=1)
    codes = one_head(blocks, P, d, 2, 118)
    q = torch.randn(n, g, d, generator=torch.Generator().manual_seed(4)).to(torch.bfloat16)
    check(form, q, codes, table, lens, [n], 0.0)


@pytest.mark.parametrize("d", (64, 128))
def test_many_rows_of_mixed_magnitude(d):
    """Rows of tiny, ordinary and huge elements, zeros, and elements far below
    their row's largest, in one unit."""
    lens, new, P, g = [90], [30], 32, 2
    table, blocks = make_tables(lens, P, seed=1)
    codes = one_head(blocks, P, d, 2, -12)
    q = torch.randn(30, g, d, generator=torch.Generator().manual_seed(4))
    q[0] *= 2.0 ** -130
    q[1] = 0
    q[2] *= torch.exp2(-torch.arange(d).float())
    q[3, 1] *= 2.0 ** 100
    q[4, 0] *= 2.0 ** 126 / q[4, 0].abs().max()
    check("many", q.to(torch.bfloat16), codes, table, lens, new, 1.0)


# ------------------------------------------------------- V scales far apart

def _apart(P, d, n_blocks, zero_scale, big_exp, seed=1):
    """Codes and table of one request: of three blocks two hold V of zeros (of
    scale ``zero_scale``) under the best keys, and one V of scale 2^big_exp
    under keys whose scores are about 132 (log2 units) below, for queries of
    ones and a scale of 1 / sqrt(d)."""
    table, blocks = make_tables([n_blocks * P], P, seed=seed)
    k8, v8, ks, vs = one_head(blocks, P, d, seed)
    gen = torch.Generator().manual_seed(seed)
    k8 = torch.randint(0x38, 0x40, k8.shape, generator=gen).to(torch.uint8)  # values 1 .. 1.875
    ks[:] = 4.0 * 8.0 / math.sqrt(d)
    for j in range(n_blocks):
        b = int(table[0, j])
        if j % 3 == 1:
            k8[b] |= 0x80
            v8[b] &= 0xEF  # magnitudes below 2^7
            vs[b] = 2.0 ** big_exp
        else:
            v8[b], vs[b] = 0, zero_scale
    return (k8, v8, ks, vs), table


@pytest.mark.parametrize("P,n_blocks", ((16, 2), (16, 50), (32, 2), (32, 40), (128, 12)))
@pytest.mark.parametrize("d", (64, 128))
@pytest.mark.parametrize("zero_scale,big_exp", ((2.0 ** -100, 14), (2.0 ** -100, 40), (2.0 ** -100, 100),
                                                (2.0 ** -100, 120), (0.0, 8), (0.0, 90), (1.0, 120)))
@pytest.mark.parametrize("form", FORMS)
def test_values_of_very_different_scale(form, zero_scale, big_exp, d, P, n_blocks):
    """Blocks of zeros under the best keys beside blocks of large values far
    below in score, which make up the whole result."""
    g, n = FORMS[form]
    codes, table = _apart(P, d, n_blocks, zero_scale, big_exp)
    q = torch.ones(n, g, d, dtype=torch.bfloat16)
    check(form, q, codes, table, [n_blocks * P], [n], 1 / math.sqrt(d), what=f"2^{big_exp}")


@pytest.mark.parametrize("d", (64, 128))
@pytest.mark.parametrize("zero_scale,big_exp", ((2.0 ** -100, 14), (2.0 ** -100, 110), (0.0, 8)))
@pytest.mark.parametrize("form", FORMS)
def test_masked_values_of_very_different_scale(form, zero_scale, big_exp, d):
    """Rows that see a block of zeros only, beside rows that see a key of a
    block of large values in the same tile as well."""
    g, n = FORMS[form]
    P = 16
    codes, table = _apart(P, d, 2, zero_scale, big_exp)
    q = torch.ones(n, g, d, dtype=torch.bfloat16)
    check(form, q, codes, table, [P + n - 2], [n], 1 / math.sqrt(d), what=f"2^{big_exp}")


# --------------------------------------------- scores near the ends of fp32's

@pytest.mark.parametrize("exp", (101, 110, 124))
@pytest.mark.parametrize("sign", (-1, 1))
@pytest.mark.parametrize("d", (64, 128))
@pytest.mark.parametrize("form", FORMS)
def test_scores_of_any_size(form, d, sign, exp):
    """One key, or equal ones, with a score of +-2^exp: L is that score (plus
    ln n) and O their values' mean.  All weights are equal, so O is off by
    their rounding to f16, the sums (2^-18) and bf16's rounding only."""
    g, n = FORMS[form]
    P = 32
    lens, new = [1, 1, 5, 70], [1, 0, n, n]
    table, blocks = make_tables(lens, P, seed=1)
    k8, v8, ks, vs = one_head(blocks, P, d, 2)
    k8[:] = 0x38  # 1.0
    T, g = sum(new), 30 if form == "many" else g  # (rows of four requests)
    q = torch.full((T, g, d), sign * 2.0 ** (exp - 6), dtype=torch.bfloat16)
    scale = 64.0 / d / float(ks[0, 0])
    o, lse, cu = attend(form, q, (k8, v8, ks, vs), table, lens, new, scale)
    O, L, A, _, _, _ = oracle.attention_cache(q, k8.numpy(), v8.numpy(), ks.numpy(), vs.numpy(), table.numpy(), lens, cu,
                                              scale, True)
    o, lse = o.cpu().double(), lse.cpu().double()
    # the score: 64 equal terms of a power of two, times log2 e and back, each rounded
    assert ((lse - L).abs() <= 2.0 ** -21 * L.abs()).all()
    bound = (2.0 ** -11 + 2.0 ** -18) * A
    assert ((o - O).abs() <= bound + 2.0 ** -8 * (O.abs() + bound)).all()


# ------------------------------------------------------- what is out of range

@pytest.mark.parametrize("bad", (-1.0, -2.0 ** -90, math.nan, math.inf, -math.inf, 2.0 ** 121, 3.4e38))
@pytest.mark.parametrize("which", ("k_scale", "v_scale"))
@pytest.mark.parametrize("P", (16, 64))
@pytest.mark.parametrize("form", FORMS)
def test_scales_out_of_range_hide_their_block(form, P, which, bad):
    """A scale that is negative, not finite or above 2^120 is reported, and its
    block's tokens are not seen, by either kernel."""
    g, n = FORMS[form]
    d, lens = 64, [5 * P + 3]
    table, blocks = make_tables(lens, P, seed=1)
    k8, v8, ks, vs = one_head(blocks, P, d, 2, -8)
    q = torch.randn(n, g, d, generator=torch.Generator().manual_seed(4)).to(torch.bfloat16)
    broken = {"k_scale": ks.clone(), "v_scale": vs.clone()}
    broken[which][int(table[0, 1])] = bad
    broken[which][int(table[0, 4])] = bad
    o, lse, cu = attend(form, q, (k8, v8, broken["k_scale"], broken["v_scale"]), table, lens, [n], 0.125, raises=614)
    rest = torch.tensor([[int(table[0, j]) for j in (0, 2, 3, 5)]], dtype=torch.int32)
    assert_forward(o, lse, q, (k8, v8, ks, vs), rest, [lens[0] - 2 * P], cu, 0.125, True, form)


@pytest.mark.parametrize("entry", (-1, -2, -5, -2 ** 31, 2 ** 31 - 1, None))
@pytest.mark.parametrize("form", FORMS)
def test_table_entries_out_of_range_hide_their_block(form, entry):
    """Any number that is no block's (None: the one behind the last block's),
    alone in a table, is reported and its tokens are not seen."""
    g, n = FORMS[form]
    d, P, lens = 64, 16, [83]
    table, blocks = make_tables(lens, P, seed=1)
    codes = one_head(blocks, P, d, 2, -8)
    q = torch.randn(n, g, d, generator=torch.Generator().manual_seed(4)).to(torch.bfloat16)
    wrong = table.clone()
    wrong[0, 2] = blocks if entry is None else entry
    o, lse, cu = attend(form, q, codes, wrong, lens, [n], 0.125, raises=611)
    rest = table[:, [0, 1, 3, 4, 5]]
    assert_forward(o, lse, q, codes, rest, [lens[0] - P], cu, 0.125, True, form)


@pytest.mark.parametrize("P", (16, 64))
@pytest.mark.parametrize("form", ("few", "many"))
def test_refused_requests_are_not_attended(form, P):
    """A request that cache_slots refuses keeps its length, and its rows their
    place: with the slot map the forward gives them no keys, where their
    positions would be those of older tokens.  The others are as ever."""
    d, H, g, R = 64, 2, 2, 4
    # table width; new tokens and the refused requests of each step
    M, steps = {"few": (2, (([5, 2 * P, 7, 2 * P - 1], []), ([1, 1, 2, 1], [1]), ([2, 3, 1, 1], [1, 3]))),
                "many": (8, (([65, 60, 7, 60], []), ([1, 8 * P, 2, 1], [1]), ([60, 1, 8 * P, 1], [2])))}[form]
    cache = fa.cache_alloc_e4m3(20, H, P, d)
    table = torch.full((R, M), -1, dtype=torch.int32, device=DEV)
    free = i32(list(range(20)))
    gen = torch.Generator().manual_seed(P)

    def rows(T, heads):
        return torch.randn(T, heads, d, generator=gen).to(torch.bfloat16)

    lens, used = i32([0] * R), i32([0])
    for step, (new, refused) in enumerate(steps):
        T = sum(new) + 2  # two rows of no request
        before = lens.tolist()
        cu, slots, lens, used = fa.cache_slots(table, lens, i32(new), free, used, P, T)
        assert [r for r in range(R) if lens[r] == before[r]] == refused
        fa.cache_append_e4m3(rows(T, H).to(DEV), rows(T, H).to(DEV), cache, slots)
        q = rows(T, H * g)
        if step > 0:
            assert_takes("few8" if form == "few" else "many", R, T, H * g, H, d)
        o, lse = fa.cache_forward_e4m3(q.to(DEV), cache, table, lens, cu, slot_map=slots)
        fa.check_errors()
        codes = [cache[i].cpu() for i in range(4)]
        c = cu.tolist()
        for r in range(R):
            at = slice(c[r], c[r + 1])
            if r in refused:
                assert (o[at] == 0).all() and (lse[at] == -math.inf).all(), f"step {step} request {r}"
            else:
                assert_forward(o[at], lse[at], q[at], codes, table[r:r + 1].cpu(), [int(lens[r])], [0, new[r]],
                               d ** -0.5, True, f"step {step} request {r}")


def test_a_slot_map_of_the_wrong_kind_is_refused():
    cache = fa.cache_alloc_e4m3(2, 1, 16, 64)
    q = torch.zeros(3, 1, 64, dtype=torch.bfloat16, device=DEV)
    args = (q, cache, i32([[0, 1]]), i32([5]), i32([0, 3]))
    with pytest.raises(TypeError, match="slot_map"):
        fa.cache_forward_e4m3(*args, slot_map=i32([0, 1, 2]))
    with pytest.raises(ValueError, match="slot_map"):
        fa.cache_forward_e4m3(*args, slot_map=torch.zeros(4, dtype=torch.int64, device=DEV))
    with pytest.raises(ValueError, match="slot_map"):
        fa.cache_forward_e4m3(*args, slot_map=torch.zeros(3, dtype=torch.int64))
    # results over the slot map, by the C entry
    slots, lse = torch.zeros(3, dtype=torch.int64, device=DEV), torch.zeros(3, 1, device=DEV)
    o, ws = torch.zeros_like(q), torch.empty(fa.cache_forward_workspace_size(1, 3, 1, 1, 64), dtype=torch.uint8, device=DEV)
    for out, l2, work in ((slots, lse, ws), (o, slots, ws), (o, lse, slots)):
        assert fa.load_library().fa_cache_fwd_e4m3_slots(
            q.data_ptr(), 64, *(c.data_ptr() for c in cache), *(t.data_ptr() for t in args[2:]), slots.data_ptr(),
            out.data_ptr(), l2.data_ptr(), 1, 3, 1, 1, 64, 2, 16, 2, 0.125, 1, work.data_ptr(), ws.numel(), None) == -1


# -------------------------------------------------------- slots at the ends

def test_slots_of_lengths_near_2_to_the_31():
    """A request whose length would pass int32 is refused, one just below is served."""
    P, M = 128, (1 << 24) + 1
    for length, new, served in ((2 ** 31 - 15, 10, True), (2 ** 31 - 11, 10, True), (2 ** 31 - 10, 10, False),
                                (2 ** 31 - 5, 10, False), (2 ** 31 - 1, 1, False), (2 ** 31 - 1, 0, True)):
        table = torch.zeros(1, M, dtype=torch.int32, device=DEV)
        table[0, (1 << 24) - 1] = 7
        cu, slots, lens, used = fa.cache_slots(table, i32([length]), i32([new]), i32([5]), i32([0]), P, 12)
        fa.check_errors()
        first = 7 * P + length % P
        want = [first + i if served and i < new else -1 for i in range(12)]
        assert slots.tolist() == want and cu.tolist() == [0, new], (length, new)
        assert lens.item() == length + (new if served else 0) and used.item() == 0, (length, new)
        assert int(table[0, -1]) == 0


def test_slots_refuse_a_map_beyond_int32():
    args = (torch.zeros(1, 4, dtype=torch.int32, device=DEV), i32([0]), i32([1]), i32([5]), i32([0]), 16)
    for tokens in (2 ** 31, 2 ** 32 + 5, -1):
        with pytest.raises(ValueError, match="num_tokens"):
            fa.cache_slots(*args, tokens)


# ------------------------------------------------ the many-row kernel's batches

@pytest.mark.parametrize("d", (64, 128))
@pytest.mark.parametrize("n", (30, 70))
def test_many_rows_some_not_finite(d, n):
    """Query rows of NaNs and of infinities leave the others as they are, with
    rows for one half of a unit and for both."""
    lens, P, g = [100, 300], 32, 2
    table, blocks = make_tables(lens, P, seed=1)
    codes = one_head(blocks, P, d, 2, -8)
    q = torch.randn(2 * n, g, d, generator=torch.Generator().manual_seed(g)).to(torch.bfloat16)
    bad = q.clone()
    where = [(0, 0), (3, 1), (n - 1, 0), (n + 5, 1), (2 * n - 1, 1)]
    for i, (t, h) in enumerate(where):
        bad[t, h] = (math.nan, math.inf, -math.inf)[i % 3]
    o, lse, cu = attend("many", bad, codes, table, lens, [n, n], 0.125)
    keep = torch.ones(2 * n, g, dtype=torch.bool)
    for t, h in where:
        keep[t, h] = False
    ref = oracle.attention_cache(q, *(c.numpy() for c in codes), table.numpy(), lens, cu, 0.125, True)
    good = ref[0].clone().to(o.dtype), ref[1].clone().to(lse.dtype)
    o, lse = o.cpu(), lse.cpu()
    o[~keep], lse[~keep] = good[0][~keep], good[1][~keep]
    assert_forward(o, lse, q, codes, table, lens, cu, 0.125, True, f"d={d} n={n}")


@pytest.mark.parametrize("P", (16, 64, 128))
@pytest.mark.parametrize("d,n", ((64, 30), (128, 70)))
def test_many_rows_report_what_is_out_of_range(d, n, P):
    """Blocks outside the cache hide their keys; lengths and rows are cut off."""
    lens, g = [6 * P + 5, n + 3], 2
    table, blocks = make_tables(lens, P, seed=1)
    codes = one_head(blocks, P, d, 2, -8)
    q = torch.randn(2 * n, g, d, generator=torch.Generator().manual_seed(4)).to(torch.bfloat16)
    q1, t1 = q[n:], table[1:]
    wrong = table.clone()
    wrong[0, 2], wrong[0, 5] = blocks, -5
    o, lse, cu = attend("many", q, codes, wrong, lens, [n, n], 0.125, causal=False, raises=611)
    rest = torch.tensor([[int(table[0, j]) for j in (0, 1, 3, 4, 6)]], dtype=torch.int32)
    assert_forward(o[:n], lse[:n], q[:n], codes, rest, [lens[0] - 2 * P], [0, n], 0.125, False)
    assert_forward(o[n:], lse[n:], q1, codes, t1, lens[1:], [0, n], 0.125, False)
    o, lse, _ = attend("many", q, codes, table, [-3, lens[1]], [n, n], 0.125, raises=612)
    assert (o[:n] == 0).all() and (lse[:n] == -math.inf).all()
    assert_forward(o[n:], lse[n:], q1, codes, t1, lens[1:], [0, n], 0.125, True)
    M = table.shape[1]
    full = torch.arange(M, dtype=torch.int32).remainder(blocks)[None]
    o, lse, _ = attend("many", q[:n], codes, full, [M * P + 5], [n], 0.125, raises=612)
    assert_forward(o, lse, q[:n], codes, full, [M * P], [0, n], 0.125, True)
    o, lse, _ = attend("many", q[:n], codes, table[1:], lens[1:], [2 * n], 0.125, causal=False, raises=613)
    assert_forward(o, lse, q[:n], codes, t1, lens[1:], [0, n], 0.125, False)


@pytest.mark.parametrize("R", (513, 1100))
def test_many_rows_of_more_requests_than_threads(R):
    """Several requests a thread in the sums, some without rows or keys."""
    P, d, g = 16, 64, 2
    gen = torch.Generator().manual_seed(R)
    new = torch.randint(0, 30, (R,), generator=gen).tolist()
    lens = [0 if i % 97 == 5 else n + int(x) for i, (n, x) in
            enumerate(zip(new, torch.randint(0, 20, (R,), generator=gen)))]
    table, blocks = make_tables(lens, P, seed=1)
    codes = one_head(blocks, P, d, 2, -8)
    poison(codes[0], table, lens)
    poison(codes[1], table, lens)
    q = torch.randn(sum(new), g, d, generator=gen).to(torch.bfloat16)
    check("many", q, codes, table, lens, new, 0.125)


@pytest.mark.parametrize("P,d", ((16, 64), (64, 128)))
def test_a_run_of_prompts(P, d):
    """Prompts, their next chunks, drafts of one request among them, one
    refused for want of blocks: slots, appends and attention together."""
    H, g, R, M = 2, 2, 3, 16
    blocks = -(-600 // P)
    gen = torch.Generator().manual_seed(P)
    free = torch.randperm(blocks, generator=gen).tolist()
    cache = fa.cache_alloc_e4m3(blocks, H, P, d)
    ref = [t.cpu().numpy() for t in cache]
    table = torch.full((R, M), -1, dtype=torch.int32, device=DEV)
    lens, used = i32([0] * R), i32([0])
    rtable, rlens, rused = table.tolist(), [0] * R, 0
    for step, new in enumerate(([90, 170, 0], [100, 3, 120], [70, 1, 16 * P], [60, 33, 65])):
        T = sum(new) + 3
        cu, slots, lens, used = fa.cache_slots(table, lens, i32(new), i32(free), used, P, T)
        rtable, rcu, rslots, rlens, rused = oracle.cache_slots(rtable, rlens, new, free, rused, P, T)
        assert table.tolist() == rtable and slots.tolist() == rslots and lens.tolist() == rlens
        k, v, q = (torch.randn(T, h, d, generator=gen).to(torch.bfloat16) for h in (H, H, H * g))
        fa.cache_append_e4m3(k.to(DEV), v.to(DEV), cache, slots)
        oracle.cache_append(k.float().numpy(), ref[0], ref[2], rslots, P)
        oracle.cache_append(v.float().numpy(), ref[1], ref[3], rslots, P)
        assert_takes("many", R, T, H * g, H, d)
        o, lse = fa.cache_forward_e4m3(q.to(DEV), cache, table, lens, cu, slot_map=slots)
        fa.check_errors()
        for a, b in zip(cache, ref):
            assert torch.equal(a.cpu(), torch.from_numpy(b)), f"step {step}"
        seen = [n if any(s >= 0 for s in rslots[rcu[r]:rcu[r + 1]]) else 0 for r, n in enumerate(rlens)]
        assert_forward(o, lse, q, [torch.from_numpy(a) for a in ref], table.cpu(), seen, rcu, d ** -0.5, True,
                       f"step {step}")
