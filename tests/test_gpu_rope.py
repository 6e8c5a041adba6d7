"""Rotary positions on the GPU against the float64 oracle, to the bit: the
result is the exact value rounded once."""
import pytest
import torch

import exact_attention_forward_04_gb300 as fa
import oracle
from exact_attention_forward_04_gb300.inputs import make_qkv

pytestmark = pytest.mark.gpu

DEV = "cuda"


def rows(*shape, seed=0, low=-6, high=6):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(*shape, generator=g) * torch.exp2(torch.randint(low, high + 1, (*shape[:-1], 1), generator=g).float())
    return x.to(torch.bfloat16)


def places(n, length, seed=0):
    g = torch.Generator().manual_seed(seed + 99)
    return torch.randint(0, length, (n,), generator=g, dtype=torch.int32)


def same(got, want, what=""):
    got, want = got.cpu(), want.cpu()
    assert got.shape == want.shape and got.dtype == want.dtype, what
    # by value, NaN alike (a zero's sign is not part of it)
    ok = (got == want) | (got.isnan() & want.isnan())
    assert ok.all(), f"{what}: {int((~ok).sum())} of {ok.numel()} differ"


@pytest.mark.parametrize("interleaved", (False, True))
@pytest.mark.parametrize("d,rot", [(64, r) for r in (16, 32, 48, 64)] + [(128, r) for r in (16, 48, 64, 112, 128)])
@pytest.mark.parametrize("T,H", ((1, 1), (3, 5), (130, 12)))
def test_tokens(d, rot, interleaved, T, H):
    table = fa.rope_table(5000, rot)
    x, pos = rows(T, H, d, seed=T + rot), places(T, 5000, seed=rot)
    got = fa.rope(x.to(DEV), pos.to(DEV), table, interleaved=interleaved)
    back = fa.rope_backward(x.to(DEV), pos.to(DEV), table, interleaved=interleaved)
    fa.check_errors()
    same(got, oracle.rope(x, pos[:, None].numpy(), table, interleaved), "rope")
    same(back, oracle.rope(x, pos[:, None].numpy(), table, interleaved, True), "rope_backward")


@pytest.mark.parametrize("interleaved", (False, True))
@pytest.mark.parametrize("own_positions", (False, True))
def test_batches(interleaved, own_positions):
    B, H, N, d, rot = 3, 2, 37, 64, 32
    table = fa.rope_table(300, rot, factor=2.0, original_length=100, magnitude=1.07)
    x = rows(B, N, H, d, seed=5).transpose(1, 2)  # as a projection leaves it
    pos = places(B * N, 300).reshape(B, N) if own_positions else places(N, 300)
    at = (pos[:, None] if own_positions else pos).numpy()
    got = fa.rope(x.to(DEV), pos.to(DEV), table, interleaved=interleaved)
    assert got.is_contiguous()
    same(got, oracle.rope(x, at, table, interleaved))
    out = torch.full((B, N, H + 1, d), 7.0, dtype=torch.bfloat16, device=DEV)
    r = fa.rope_backward(x.to(DEV), pos.to(DEV), table, interleaved=interleaved, out=out[:, :, :H].transpose(1, 2))
    fa.check_errors()
    same(r, oracle.rope(x, at, table, interleaved, True))
    assert (out[:, :, H] == 7).all()


def test_many_values_next_to_borders():
    """Enough values that thousands lie where a fp32 sum cannot tell their
    rounding, and pairs that cancel to far below their terms; checked in 64
    bits on the GPU, pair by pair."""
    T, H, d = 4000, 16, 128
    table = fa.rope_table(70000, d)
    pos = places(T, 70000).to(DEV)
    x = rows(T, H, d, seed=3, low=0, high=0).to(DEV)
    c, s = (table[pos.long()][..., i].double()[:, None] for i in (0, 1))
    x[: T // 2, :, d // 2:] = (x[: T // 2, :, :d // 2].double() * c[: T // 2] / s[: T // 2]).to(torch.bfloat16)
    y = fa.rope(x, pos, table)
    a, b = x[..., :d // 2].double(), x[..., d // 2:].double()
    want = torch.cat((a * c - b * s, b * c + a * s), -1)
    step = torch.exp2(torch.floor(torch.log2(want.abs().clamp(min=2.0 ** -120))) - 7)
    assert torch.equal(y.double(), torch.round(want / step) * step)


def test_infinities_nan_and_extremes():
    """They go through their own pair's formula and no other's."""
    table = fa.rope_table(50, 64)
    x = rows(6, 1, 64, seed=1)
    big = 3.3895313892515355e38
    x[0, 0, 3], x[1, 0, 40], x[2, 0, 5], x[3, 0, 0], x[4, 0, 1] = float("inf"), -float("inf"), float("nan"), big, 1e-40
    x[5, 0, 2], x[5, 0, 34] = big, -big
    pos = torch.tensor([7, 7, 7, 0, 1, 9], dtype=torch.int32)
    got = fa.rope(x.to(DEV), pos.to(DEV), table)
    fa.check_errors()
    same(got, oracle.rope(x, pos[:, None].numpy(), table))


@pytest.mark.parametrize("interleaved", (False, True))
@pytest.mark.parametrize("rot", (48, 128))
def test_in_place_slices_and_broadcast_rows(interleaved, rot):
    T, H, d = 70, 6, 128
    table, pos = fa.rope_table(200, rot), places(T, 200)
    qkv = rows(T, H + 4, d, seed=2)
    want = oracle.rope(qkv[:, :H], pos[:, None].numpy(), table, interleaved)
    t = qkv.to(DEV)
    r = fa.rope(t[:, :H], pos.to(DEV), table, interleaved=interleaved, out=t[:, :H])
    assert r.data_ptr() == t.data_ptr()
    same(t[:, :H], want)
    same(t[:, H:], qkv[:, H:])
    one = qkv[:, :1].to(DEV).expand(T, 5, d)  # one row for all heads
    same(fa.rope(one, pos.to(DEV), table, interleaved=interleaved),
         oracle.rope(qkv[:, :1], pos[:, None].numpy(), table, interleaved).expand(T, 5, d))
    fa.check_errors()


def test_positions_outside_the_table():
    """Negative: copied. Beyond: copied and reported."""
    table = fa.rope_table(20, 32)
    x = rows(4, 3, 64, seed=9)
    pos = torch.tensor([-1, 19, -2 ** 31, 3], dtype=torch.int32)
    same(fa.rope(x.to(DEV), pos.to(DEV), table), oracle.rope(x, pos[:, None].numpy(), table))
    fa.check_errors()
    for far in (20, 2 ** 31 - 1):
        pos[0] = far
        y = fa.rope(x.to(DEV), pos.to(DEV), table)
        with pytest.raises(fa.FAError) as e:
            fa.check_errors()
        assert e.value.status == -6 and "site=621" in str(e.value)
        same(y, oracle.rope(x, pos[:, None].numpy(), table))


def test_nothing_and_refusals():
    table = fa.rope_table(20, 32)
    x, none = rows(4, 3, 64).to(DEV), torch.zeros(0, dtype=torch.int32, device=DEV)
    assert fa.rope(x[:0], none, table).shape == (0, 3, 64)
    pos = torch.zeros(4, dtype=torch.int32, device=DEV)
    for bad in (dict(positions=pos.long()), dict(positions=pos[:3]), dict(table=table.double()), dict(x=x[..., ::2]),
                dict(table=table[:, :4].contiguous()), dict(x=x.float()), dict(out=torch.empty_like(x[:2])),
                dict(table=table[:, :, :1].contiguous()), dict(positions=pos.cpu())):
        a = dict(x=x, positions=pos, table=table)
        a.update(bad)
        with pytest.raises((TypeError, ValueError)):
            fa.rope(**a)
    with pytest.raises(fa.FAError):   # neither in place nor apart
        fa.rope(x[:3], pos[:3], table, out=x[1:])
    with pytest.raises(fa.FAError):   # rows of out that share memory
        fa.rope(x, pos, table, out=torch.zeros(4, 1, 64, dtype=torch.bfloat16, device=DEV).expand(4, 3, 64))


def test_more_than_4_gib():
    n = (1 << 31) // 64 + 100
    x = torch.zeros(1, 1, n, 64, dtype=torch.bfloat16, device=DEV)
    x[0, 0, -50:] = rows(50, 64, seed=4).to(DEV)
    table = fa.rope_table(128, 64)
    pos = (torch.arange(n, device=DEV) % 128).int()
    y = fa.rope(x, pos, table)
    fa.check_errors()
    same(y[0, 0, -50:], oracle.rope(x[0, 0, -50:], pos[-50:].cpu().numpy(), table))


def test_gradient_through_attention():
    """Queries and keys turned, attended, and the gradients turned back: against
    the oracle's gradients of the turned rows, and against differences."""
    B, H, N, d = 1, 2, 70, 64
    q, k, v = make_qkv(B, H, N, d, seed=11)
    g = make_qkv(B, H, N, d, seed=12)[0]
    table, pos = fa.rope_table(N, d), torch.arange(N, dtype=torch.int32)
    t, p = table.to(DEV), pos.to(DEV)
    qr, kr = (fa.rope(x.to(DEV), p, t) for x in (q, k))
    o, lse = fa.forward(qr, kr, v.to(DEV), causal=True)
    dqr, dkr, dv = fa.backward(qr, kr, v.to(DEV), o, lse, g.to(DEV), causal=True)
    dq, dk = (fa.rope_backward(x, p, t) for x in (dqr, dkr))
    fa.check_errors()
    same(dq, oracle.rope(dqr, pos.numpy(), table, False, True))
    same(dk, oracle.rope(dkr, pos.numpy(), table, False, True))
    # the loss sum(o g) in 64 bits, along a direction of q and of k
    rot = lambda x: torch.from_numpy(oracle.rotate(x.numpy(), pos.numpy(), table.cpu().numpy()))  # noqa: E731
    gen = torch.Generator().manual_seed(13)

    def loss(a, b):
        return (oracle.attention_ref(rot(a), rot(b), v, d ** -0.5, True)[0] * g.double()).sum().item()

    for which, grad in ((0, dq), (1, dk)):
        e = torch.randn(q.shape, generator=gen, dtype=torch.float64)
        h = 1e-5
        x = [q.double(), k.double()]
        hi, lo = list(x), list(x)
        hi[which], lo[which] = x[which] + h * e, x[which] - h * e
        slope = (loss(*hi) - loss(*lo)) / (2 * h)
        terms = grad.cpu().double() * e
        # each gradient element is a bf16 of the attention's backward (off by 2e-2 of
        # the largest at most, as its tests hold) turned and rounded: errors of
        # independent signs add up like the root of their number
        bound = 2e-2 * grad.abs().max().item() * e.norm().item() * 4
        assert abs(terms.sum().item() - slope) < bound


def test_streams_and_graphs():
    table = fa.rope_table(900, 128)
    T, H, d = 33, 4, 128
    x, pos = rows(T, H, d, seed=1).to(DEV), places(T, 900).to(DEV)
    want = fa.rope(x, pos, table)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for stream in (s, s.cuda_stream):
        got = fa.rope(x, pos, table, stream=stream)
        s.synchronize()
        same(got, want)
    xs, ps = x.clone(), pos.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = fa.rope(xs, ps, table)
        z = fa.rope_backward(y, ps, table)
    for i in range(3):
        xs.copy_(rows(T, H, d, seed=20 + i))
        ps.copy_(places(T, 900, seed=i))
        graph.replay()
        same(y, fa.rope(xs, ps, table))
        same(z, fa.rope_backward(y, ps, table))
    fa.check_errors()
