"""Rotary positions where one rounding of the exact value is hard to come by:
pairs that cancel, small numbers, ties that a far smaller term decides.  To the
bit, against the oracle, which tests/test_oracle_rope.py pins with rationals."""
import numpy as np
import pytest
import torch

import exact_attention_forward_04_gb300 as fa
import oracle

pytestmark = pytest.mark.gpu

DEV = "cuda"
F = np.float32


def same(got, want, what=""):
    got, want = got.cpu(), want.cpu()
    assert got.shape == want.shape and got.dtype == want.dtype, what
    ok = (got == want) | (got.isnan() & want.isnan())   # a zero's sign is not part of it
    assert ok.all(), f"{what}: {int((~ok).sum())} of {ok.numel()} differ, first at {(~ok).nonzero()[:3].tolist()}"


def laid(a, b, d, interleaved):
    """Pairs a, b [T, n] (bf16 values) as rows [T, 1, d], zeros behind them."""
    T, n = a.shape
    x = np.zeros((T, d))
    if interleaved:
        x[:, 0:2 * n:2], x[:, 1:2 * n:2] = a, b
    else:
        x[:, :n], x[:, n:2 * n] = a, b
    t = torch.from_numpy(x).to(torch.bfloat16)
    assert (t.double().numpy() == x).all()
    return t[:, None]


def check(a, b, table, pos=None, d=128):
    """rope and rope_backward of pairs a, b [T, n] at ``pos`` (row t of the table for row t)."""
    table = torch.as_tensor(table)
    assert table.dtype == torch.float32
    pos = torch.arange(a.shape[0]) if pos is None else torch.as_tensor(pos)
    pos, t = pos.int(), table.to(DEV)
    for interleaved in (False, True):
        x = laid(a, b, d, interleaved)
        got = fa.rope(x.to(DEV), pos.to(DEV), t, interleaved=interleaved)
        back = fa.rope_backward(x.to(DEV), pos.to(DEV), t, interleaved=interleaved)
        fa.check_errors()
        at = pos[:, None].numpy()
        same(got, oracle.rope(x, at, table, interleaved), f"rope, interleaved={interleaved}")
        same(back, oracle.rope(x, at, table, interleaved, True), f"rope_backward, interleaved={interleaved}")


def mantissas(g, *shape):
    return g.integers(128, 256, shape) / 128.0


def doubtful(c, s):
    """A pair in [1, 2) whose first result lies so near a border of bf16's rounding that a fp32 sum cannot tell."""
    x, y = (np.arange(128, 256) / 128.0 for _ in range(2))
    r = (x[:, None] * float(c) - y * float(s)).astype(F)
    low = r.view(np.uint32) & 0xffff
    at = np.argwhere((low >= 0x7fff) & (low <= 0x8001))
    return (x[at[0][0]], y[at[0][1]]) if len(at) else None


CANCEL = ((27076, 53, 1.0625, 1.4921875), (30391, 19, 1.0, 1.4140625), (2638, 59, 1.0625, 1.765625))


@pytest.mark.parametrize("neighbour", (False, True))
@pytest.mark.parametrize("pos,i,x,y", CANCEL)
def test_pairs_that_cancel_in_a_plain_table(pos, i, x, y, neighbour):
    """The rounded products are the same number, and what their roundings lost is the
    result; with and without a pair beside it that is taken again."""
    table = fa.rope_table(32768, 128, device="cpu")
    a, b = np.zeros((4, 64)), np.zeros((4, 64))
    for r, (p, q) in enumerate(((x, y), (y, -x), (-x, -y), (y, x))):   # the last does not cancel, but its gradient does
        a[r, i], b[r, i] = p, q
    if neighbour:
        for j in range(i // 8 * 8, i // 8 * 8 + 8):
            two = doubtful(*table[pos, j].tolist()) if j != i else None
            if two:
                a[:, j], b[:, j] = two
                break
        else:
            pytest.fail("no pair next to a border")
    check(a, b, table, [pos] * 4)


def cancelling(g, T, n, scale=1.0):
    """Pairs a, b [T, n] and a table [T, n, 2] with RN(a c) = RN(b s), the exact difference mostly not 0."""
    a, b = mantissas(g, T, n), mantissas(g, T, n) * 2.0 ** g.integers(-3, 4, (T, n))
    b *= np.where(g.random((T, n)) < 0.5, -1, 1)
    s = g.uniform(0.25, 1, (T, n)).astype(F)
    c = (b * s / a).astype(F)
    for _ in range(4):  # where a product misses, the entry beside may hit
        p, q = (a.astype(F) * c), (b.astype(F) * s)
        c = np.where(p == q, c, np.nextafter(c, np.where(p < q, F(np.inf), F(-np.inf)))).astype(F)
    hit = (a.astype(F) * c) == (b.astype(F) * s)
    exact = a * c.astype(float) - b * s.astype(float)
    assert hit.mean() > 0.5 and (exact[hit] != 0).mean() > 0.9
    return np.where(hit, a, 0) * scale, np.where(hit, b, 0) * scale, np.stack((c, s), -1)


@pytest.mark.parametrize("scale", (1.0, 2.0 ** -40, 2.0 ** -70, 2.0 ** 90))
def test_pairs_that_cancel(scale):
    g = np.random.default_rng(5)
    a, b, table = cancelling(g, 300, 64, scale)
    a[1::2, ::8], b[1::2, ::8] = scale, 0                     # 1 + 2^-8, a tie, in every lane of every other row
    table[1::2, ::8] = 257 / 256, 0.5
    check(a, b, table)


def test_append_turns_cancelling_pairs_to_the_same_bits():
    """Groups of nothing but rests of about 2^-25, some of them beside a tie."""
    g = np.random.default_rng(6)
    T, d = 200, 128
    a, b, table = cancelling(g, T, 64)
    a[1::2, ::8], b[1::2, ::8] = 2.0 ** -25, 0
    table[1::2, ::8] = 257 / 256, 0.5
    table, pos = torch.from_numpy(table), torch.arange(T, dtype=torch.int32)
    slots = torch.arange(T, device=DEV)
    for interleaved in (False, True):
        k = laid(a, b, d, interleaved)
        one, two = (fa.cache_alloc_e2m1(T // 16 + 1, 1, 16, d, k_unit=2.0 ** -30) for _ in range(2))
        fa.cache_append_e2m1(k.to(DEV), k.to(DEV), one, slots, positions=pos.to(DEV), table=table.to(DEV),
                             interleaved=interleaved)
        turned = oracle.rope(k, pos[:, None].numpy(), table, interleaved)
        fa.cache_append_e2m1(turned.to(DEV), k.to(DEV), two, slots)
        fa.check_errors()
        assert torch.equal(one.data, two.data)
        assert (fa.cache_read_e2m1(one, slots)[0] != 0).float().mean() > 0.2


@pytest.mark.parametrize("d", (64, 128))
def test_rows_of_small_numbers(d):
    """Subnormals of bf16 and what lies just above, alone in their rows: at position
    0, where they come back as they are, and turned; and beside pairs taken again."""
    g = np.random.default_rng(7)
    n, T = d // 2, 240
    table = fa.rope_table(4000, d, device="cpu")
    low = np.repeat(np.arange(-133, -85), 5)[:, None]                       # a row's smallest step
    a, b = (g.integers(-255, 256, (T, n)) * 2.0 ** np.maximum(low, -133) for _ in range(2))
    check(a, b, table, [0] * T, d)
    same(fa.rope(laid(a, b, d, False).to(DEV), torch.zeros(T, dtype=torch.int32, device=DEV), table.to(DEV)),
         laid(a, b, d, False))
    check(a, b, table, g.integers(0, 4000, T), d)
    table = table.clone()
    table[::2, ::8] = torch.tensor([257 / 256, 0.0])
    a[:, ::8], b[:, ::8] = 1.0, 0.0
    check(a, b, table, g.integers(0, 4000, T), d)


def test_small_table_entries():
    """Products far below their factors, down to below fp32."""
    g = np.random.default_rng(8)
    T, n = 200, 64
    a, b = (mantissas(g, T, n) * 2.0 ** g.integers(-60, 3, (T, n)) for _ in range(2))
    table = (g.uniform(-1, 1, (T, n, 2)) * 2.0 ** g.integers(-149, 1, (T, n, 1))).astype(F)
    a[1::2, ::8], b[1::2, ::8] = 1.0, 0.0                     # a tie in every lane of every other row
    table[1::2, ::8] = 257 / 256, 0.5
    check(a, b, table)


def test_products_beyond_fp32():
    """Of the largest numbers, with entries above 1: results that fp32 holds again, results
    that nothing does, and ties, exact all of them."""
    g = np.random.default_rng(10)
    T, n = 200, 64
    a, b = (mantissas(g, T, n) * 2.0 ** g.integers(124, 128, (T, n)) * np.where(g.random((T, n)) < 0.5, -1, 1)
            for _ in range(2))
    table = g.uniform(-4, 4, (T, n, 2)).astype(F)
    near = np.arange(n) % 2 == 0                                   # a c and b s nearly the same
    table[:, near, 0] = (b * table[..., 1] / a * (1 + g.uniform(-0.1, 0.1, (T, n))))[:, near]
    table = np.clip(table, -30, 30)
    a[1::2, ::8], b[1::2, ::8] = 1.0, 0.0
    table[1::2, ::8] = 257 / 256, 0.5
    first = a * table[..., 0].astype(float) - b * table[..., 1].astype(float)
    top = np.abs(a * table[..., 0].astype(float)) > 2.0 ** 128
    assert (top & (np.abs(first) < 2.0 ** 127)).mean() > 0.1 and (np.abs(first) > 2.0 ** 128).mean() > 0.1
    check(a, b, table)


TIES = ((1.265625, 0.75390625, 0.89197528362, 4.200120073960534e-08),
        (1.0, 2.0 ** -100, 257 / 256, 2.0 ** -60))


@pytest.mark.parametrize("x,y,c,s", TIES)
def test_a_tie_and_a_term_far_below(x, y, c, s):
    a, b, table = np.zeros((8, 8)), np.zeros((8, 8)), np.zeros((8, 8, 2), F)
    rows = [(sx * p, sy * q) for p, q in ((x, y), (y, x)) for sx in (1, -1) for sy in (1, -1)]
    for r, (p, q) in enumerate(rows):
        a[r, r], b[r, r] = p, q
        table[r, r] = (c, s) if r < 4 else (s, c)
    check(a, b, table, d=64)


def test_ties_that_the_other_term_decides():
    """The first product is a tie of bf16, or fp32 rounds it to one, and the other is
    anything from a step of bf16 to nothing that fp32 holds, or takes back what that
    rounding lost, but for its last bits."""
    g = np.random.default_rng(9)
    T, n = 300, 64
    a = mantissas(g, T, n)
    tie = (2 * g.integers(128, 256, (T, n)) + 1) / 256.0
    a[: T // 3] = 1.0
    c = (tie / a).astype(F)
    b = mantissas(g, T, n) * np.where(g.random((T, n)) < 0.5, -1, 1)
    size = 2.0 ** -g.integers(8, 250, (T, n)).astype(float)
    lost = a * c.astype(float) - (a.astype(F) * c)
    back = (np.arange(T)[:, None] % 2 == 1) & (lost != 0)
    size_b = np.where(back, 1.0, np.maximum(size, 2.0 ** -120))
    b = b * size_b
    s = np.where(back, lost / b, np.minimum(size / size_b, 1.0)).astype(F)
    assert back.mean() > 0.2 and ((a.astype(F) * c).astype(float) == tie).mean() > 0.5
    check(a, b, np.stack((c, s), -1))
    check(-a, b, np.stack((c, s), -1))
