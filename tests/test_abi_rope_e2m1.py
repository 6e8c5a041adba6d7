"""Refusals of rotary positions and of the 4-bit key/value cache, on the host:
fake addresses that are never dereferenced, and CPU tensors.  And the oracle's
pins."""
import math

import numpy as np
import pytest
import torch

import exact_attention_forward_04_gb300 as fa
import oracle

FA_OK, INVALID, UNSUPPORTED, MISALIGNED = 0, -1, -2, -3


@pytest.fixture(scope="module")
def lib():
    from exact_attention_forward_04_gb300 import _build
    _build.build()
    return fa.load_library()


X, OUT, POS, TAB = (0x10000000 * (i + 1) for i in range(4))


def _rope(lib, x=X, xs=(8192, 1024, 128), out=OUT, os=(8192, 1024, 128), pos=POS, ps=0, tab=TAB, length=100, B=2, H=8,
          N=8, d=128, rot=128, il=0, tr=0):
    return lib.fa_rope(x, *xs, out, *os, pos, ps, tab, length, B, H, N, d, rot, il, tr, None)


@pytest.mark.parametrize("kw,want", [
    (dict(x=0), INVALID), (dict(out=0), INVALID), (dict(pos=0), INVALID), (dict(tab=0), INVALID),
    (dict(length=0), INVALID), (dict(B=-1), INVALID),
    (dict(H=0), INVALID), (dict(N=-1), INVALID), (dict(il=2), INVALID), (dict(tr=-1), INVALID),
    (dict(d=96), UNSUPPORTED), (dict(rot=0), UNSUPPORTED), (dict(rot=24), UNSUPPORTED), (dict(rot=144), UNSUPPORTED),
    (dict(d=64, rot=128), UNSUPPORTED), (dict(ps=7), INVALID), (dict(ps=-8), INVALID),
    (dict(xs=(8192, 1024, -128)), INVALID), (dict(os=(8192, 1024, 64)), INVALID), (dict(os=(8192, 0, 128)), INVALID),
    (dict(os=(1024, 1024, 128)), INVALID),       # rows of out that overlap
    (dict(xs=(8192, 1024, 132)), MISALIGNED), (dict(os=(8192, 1028, 128)), MISALIGNED),
    (dict(xs=(1 << 32, 1024, 128)), UNSUPPORTED), (dict(x=X + 8), MISALIGNED), (dict(out=OUT + 2), MISALIGNED),
    (dict(tab=TAB + 8), MISALIGNED), (dict(pos=POS + 1), MISALIGNED),
    (dict(out=X + 256), INVALID), (dict(out=X, os=(8192, 128, 1024)), INVALID),  # neither apart nor in place
    (dict(pos=OUT + 64), INVALID), (dict(tab=OUT + 64), INVALID),
    (dict(B=1 << 20, N=1 << 20), INVALID), (dict(B=0), FA_OK), (dict(N=0, x=0, pos=0), FA_OK),
])
def test_rope_refusals(lib, kw, want):
    assert _rope(lib, **kw) == want


K, V, DATA, SLOT = (0x10000000 * (i + 5) for i in range(4))


def _append(lib, k=K, v=V, ks=384, vs=384, data=DATA, ku=1.0, vu=0.25, slot=SLOT, pos=POS, tab=TAB, length=100, rot=64,
            il=0, T=20, H=3, d=128, blocks=10, P=32):
    return lib.fa_cache_append_e2m1(k, v, ks, vs, data, ku, vu, slot, pos, tab, length, rot, il, T, H, d, blocks, P,
                                    None)


UNITS = [dict(ku=0.0), dict(ku=-1.0), dict(vu=3.0), dict(vu=math.inf), dict(ku=math.nan), dict(ku=2.0 ** 65),
         dict(vu=2.0 ** -65)]


@pytest.mark.parametrize("kw,want", [
    (dict(k=0), INVALID), (dict(v=0), INVALID), (dict(data=0), INVALID), (dict(slot=0), INVALID),
    (dict(tab=0), INVALID), (dict(length=0), INVALID), (dict(rot=0), UNSUPPORTED), (dict(rot=72), UNSUPPORTED),
    (dict(rot=256), UNSUPPORTED), (dict(il=3), INVALID), (dict(T=-1), INVALID), (dict(H=0), INVALID),
    (dict(blocks=0), INVALID), (dict(d=96), UNSUPPORTED), (dict(P=20), UNSUPPORTED), (dict(blocks=1 << 30), UNSUPPORTED),
    (dict(ks=376), INVALID), (dict(vs=-384), INVALID), (dict(ks=388), MISALIGNED), (dict(k=K + 8), MISALIGNED),
    (dict(data=DATA + 8), MISALIGNED), (dict(slot=SLOT + 4), MISALIGNED), (dict(pos=POS + 2), MISALIGNED),
    (dict(tab=TAB + 4), MISALIGNED), (dict(k=DATA), INVALID), (dict(v=DATA + 512), INVALID),
    (dict(slot=DATA + 512), INVALID), (dict(pos=DATA), INVALID), (dict(tab=DATA), INVALID),
    (dict(T=0), FA_OK), (dict(T=0, k=0, slot=0, pos=0), FA_OK), *[(u, INVALID) for u in UNITS],
])
def test_append_refusals(lib, kw, want):
    assert _append(lib, **kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(data=0), INVALID), (dict(slot=0), INVALID), (dict(k=0), INVALID), (dict(v=0), INVALID),
    (dict(T=-1), INVALID), (dict(H=-1), INVALID), (dict(d=32), UNSUPPORTED), (dict(P=8), UNSUPPORTED),
    (dict(k=K + 4), MISALIGNED), (dict(slot=SLOT + 2), MISALIGNED), (dict(v=K + 256), INVALID),
    (dict(k=DATA + 256), INVALID), (dict(v=SLOT), INVALID), (dict(T=0, k=0), FA_OK), *[(u, INVALID) for u in UNITS],
])
def test_read_refusals(lib, kw, want):
    a = dict(data=DATA, ku=1.0, vu=1.0, slot=SLOT, k=K, v=V, T=20, H=3, d=128, blocks=10, P=32)
    a.update(kw)
    assert lib.fa_cache_read_e2m1(*a.values(), None) == want


Q, O, L, WS = 0x91000000, 0x92000000, 0x93000000, 0x94000000


@pytest.mark.parametrize("kw,want", [
    (dict(q=0), INVALID), (dict(data=0), INVALID), (dict(tab=0), INVALID), (dict(lens=0), INVALID),
    (dict(cu=0), INVALID), (dict(o=0), INVALID), (dict(lse=0), INVALID), (dict(ws=0), INVALID), (dict(R=-1), INVALID),
    (dict(T=-1), INVALID), (dict(Hq=7), INVALID), (dict(H=0), INVALID), (dict(M=0), INVALID),
    (dict(d=96), UNSUPPORTED), (dict(P=48), UNSUPPORTED), (dict(scale=math.inf), INVALID), (dict(causal=2), INVALID),
    (dict(stride=760), INVALID), (dict(stride=772), MISALIGNED), (dict(q=Q + 8), MISALIGNED),
    (dict(data=DATA + 4), MISALIGNED), (dict(slot=SLOT + 4), MISALIGNED), (dict(T=1 << 30), UNSUPPORTED),
    (dict(T=0), FA_OK), (dict(R=0), FA_OK), *[(u, INVALID) for u in UNITS],
])
def test_forward_refusals(lib, kw, want):
    a = dict(q=Q, stride=768, data=DATA, ku=1.0, vu=1.0, tab=0xA0000000, lens=0xA1000000, cu=0xA2000000, slot=0, o=O,
             lse=L, R=4, T=9, Hq=6, H=3, d=128, blocks=10, P=32, M=5, scale=0.1, causal=1, ws=WS, n=1 << 30)
    a.update(kw)
    assert lib.fa_cache_fwd_e2m1(*a.values(), None) == want


def test_slots_with_positions_refuses_none(lib):
    a = [0x10000000 * (i + 1) for i in range(10)]
    a[7] = 0
    assert lib.fa_cache_slots_positions(*a, 4, 8, 16, 32, 20, None) == INVALID
    a[7] = a[6] + 8  # over the slot map
    assert lib.fa_cache_slots_positions(*a, 4, 8, 16, 32, 20, None) == INVALID
    a[7] = 0x80000002
    assert lib.fa_cache_slots_positions(*a, 4, 8, 16, 32, 20, None) == MISALIGNED


def test_python_refuses_what_it_cannot_take():
    x, pos = torch.zeros(4, 2, 64, dtype=torch.bfloat16), torch.zeros(4, dtype=torch.int32)
    table = fa.rope_table(16, 32, device="cpu")
    with pytest.raises(ValueError, match="CUDA"):
        fa.rope(x, pos, table)
    with pytest.raises(TypeError):
        fa.rope(x.float(), pos, table)
    with pytest.raises(ValueError, match="multiple of 16"):
        fa.rope_table(16, 24, device="cpu")
    with pytest.raises(ValueError):
        fa.rope_table(0, 32, device="cpu")
    with pytest.raises(ValueError, match="CUDA"):
        fa.cache_append_e2m1(x, x, fa.CacheE2M1(torch.zeros(2, 2, 1, 18 * 64, dtype=torch.uint8)), pos.long())
    with pytest.raises(ValueError):
        fa.cache_alloc_e2m1(2, 2, 24, 64, device="cpu")
    with pytest.raises(ValueError):
        fa.cache_alloc_e2m1(2, 2, 16, 80, device="cpu")


# ------------------------------------------------------------------- pins

def test_table_angles():
    t = fa.rope_table(5000, 64, base=500.0, device="cpu").double()
    i = torch.arange(32, dtype=torch.float64)
    for p in (0, 1, 4999):
        a = p * 500.0 ** (-i / 32)
        assert torch.equal(t[p, :, 0], a.cos().float().double()) and torch.equal(t[p, :, 1], a.sin().float().double())


def test_table_scaled_for_longer_contexts():
    plain, by4 = fa.rope_table(64, 32, device="cpu"), fa.rope_table(256, 32, factor=4.0, device="cpu")
    assert torch.allclose(by4[::4], plain, atol=1e-6)          # position interpolation
    parts = fa.rope_table(256, 32, factor=4.0, original_length=64, low=1.0, high=2.0, magnitude=0.5, device="cpu")
    f = 10000.0 ** (-np.arange(16) / 16)
    turns = 64 * f / (2 * np.pi)
    for i in range(16):
        want = plain[1, i] if turns[i] >= 2 else by4[1, i] if turns[i] <= 1 else None
        if want is not None:
            assert torch.allclose(parts[1, i], 0.5 * want, atol=1e-6)
    assert (turns >= 2).any() and (turns <= 1).any()


@pytest.mark.parametrize("interleaved", (False, True))
def test_oracle_rotation(interleaved):
    """Lengths of pairs kept, products of two rows a function of their distance,
    the transposed rotation the gradient (by automatic differentiation)."""
    g = torch.Generator().manual_seed(1)
    table = fa.rope_table(64, 32, device="cpu").double().numpy()
    x, y = torch.randn(2, 64, generator=g, dtype=torch.float64).numpy()
    at = lambda v, p: oracle.rotate(v[None], [p], table, interleaved)[0]  # noqa: E731
    assert np.array_equal(at(x, 0), x) and np.array_equal(at(x, -1), x) and np.array_equal(at(x, 64), x)
    assert np.allclose(at(x, 9) @ at(y, 4), at(x, 25) @ at(y, 20), rtol=0, atol=1e-5)  # fp32 table entries
    assert np.array_equal(at(x, 9)[32:], x[32:]) and not np.allclose(at(x, 9)[:32], x[:32])
    rot = np.stack([oracle.rotate(np.eye(64), [7] * 64, table, interleaved)])[0].T   # columns: images of unit vectors
    back = oracle.rotate(y[None], [7], table, interleaved, True)[0]
    assert np.allclose(rot.T @ y, back)
    xt = torch.tensor(x, requires_grad=True)
    (torch.from_numpy(rot) @ xt @ torch.from_numpy(y)).backward()
    assert np.allclose(xt.grad.numpy(), back)


def test_oracle_round_bf16():
    g = torch.Generator().manual_seed(2)
    x = torch.randn(2000, generator=g) * torch.exp2(torch.randint(-130, 100, (2000,), generator=g).float())
    assert np.array_equal(oracle.round_bf16(x.double().numpy()), x.to(torch.bfloat16).double().numpy())
    tie = 1 + 2.0 ** -8
    assert oracle.round_bf16(tie) == 1 and oracle.round_bf16(tie + 2.0 ** -40) == 1 + 2.0 ** -7


def test_oracle_codes():
    e = oracle.cache_e2m1
    v = np.array([0, .25, .26, .75, .74, 1.25, 1.75, 2.5, 2.51, 3.5, 5, 5.01, 9, -0.3, -5])
    assert e.e2m1_decode(e.e2m1_encode(v)).tolist() == [0, 0, .5, 1, .5, 1, 2, 2, 3, 4, 4, 6, 6, -.5, -4]
    assert np.array_equal(e.e2m1_encode(e.e2m1_decode(np.arange(16))), np.arange(16))
    c, s = e.quantise(np.full((1, 16), 12.0), 0.5)    # 12 / 6 / 0.5 = 4
    assert oracle.e4m3_decode(s)[0, 0] == 4 and (c == 7).all()
    c, s = e.quantise(np.full((1, 16), 1e-9), 1.0)    # below the scales
    assert (s == 0).all() and (c == 0).all()
    c, s = e.quantise(np.full((1, 16), 1e9), 1.0)     # above
    assert oracle.e4m3_decode(s)[0, 0] == 448 and (c == 7).all()


@pytest.mark.parametrize("d", (64, 128))
def test_oracle_layout(d):
    """Every byte of 18 d belongs to one scale or to two codes."""
    for (byte, shift, scale) in oracle.cache_e2m1.places(d):
        assert len(set(zip(byte.ravel(), shift.ravel()))) == 16 * d
        assert len(set(scale.ravel())) == d
    (kb, _, ks), (vb, _, vs) = oracle.cache_e2m1.places(d)
    used = np.concatenate([np.unique(a) for a in (kb, ks, vb, vs)])
    assert np.array_equal(np.sort(used), np.arange(18 * d))
    g = np.random.default_rng(1)
    data = np.zeros((2, 1, 2, 18 * d), np.uint8)
    k, v = g.normal(size=(2, 40, 1, d))
    slots = g.permutation(64)[:40]
    oracle.cache_e2m1.append(data, k, v, slots, 0.5, 0.25)
    kk, vv = oracle.cache_e2m1.values(data, 0.5, 0.25)
    for x, y in ((k, kk), (v, vv)):
        got = y.transpose(0, 2, 1, 3).reshape(64, 1, d)[slots]
        assert np.abs(got - x).max() < 0.6 and np.linalg.norm(got - x) < 0.12 * np.linalg.norm(x)


def test_oracle_attention_agrees_with_the_dense_oracle():
    d, P, n = 64, 16, 40
    from tests.cache4_cases import make_data
    data = make_data(3, 1, P, d, 1).numpy()
    k, v = oracle.cache_e2m1.values(data, 1.0, 0.5)
    k, v = (x.transpose(0, 2, 1, 3).reshape(-1, d)[:n] for x in (k, v))
    q = torch.randn(n, 1, d, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16)
    O, L, *_ = oracle.cache_e2m1.attention(q, data, 1.0, 0.5, [[0, 1, 2]], [n], [0, n], 0.05)
    to = lambda x: torch.from_numpy(x)[None, None]  # noqa: E731
    O_ref, L_ref = oracle.attention_ref(q.transpose(0, 1)[None], to(k), to(v), 0.05, True)
    assert torch.allclose(O[:, 0], O_ref[0, 0], atol=1e-12) and torch.allclose(L[:, 0], L_ref[0, 0], atol=1e-12)
