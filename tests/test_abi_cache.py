"""Refusals of the 8-bit key/value cache's entry points, on the host: fake
addresses that are never dereferenced, and CPU tensors.  And the oracle's
pins."""
import numpy as np
import pytest
import torch

import exact_attention_forward_04_gb300 as fa
import oracle
from exact_attention_forward_04_gb300 import cache as cache_mod
from tests.cache_cases import make_codes, make_tables

FA_OK, INVALID, UNSUPPORTED, MISALIGNED = 0, -1, -2, -3


@pytest.fixture(scope="module")
def lib():
    from exact_attention_forward_04_gb300 import _build
    _build.build()
    return fa.load_library()


TAB, LEN, NEW, FREE, USED, CU, SLOT, LEN2, USED2 = (0x10000000 * (i + 1) for i in range(9))


def _slots(lib, tab=TAB, lens=LEN, new=NEW, free=FREE, used=USED, cu=CU, slot=SLOT, lens2=LEN2, used2=USED2, R=4,
           M=8, F=16, P=32, T=20):
    return lib.fa_cache_slots(tab, lens, new, free, used, cu, slot, lens2, used2, R, M, F, P, T, None)


@pytest.mark.parametrize("kw,want", [
    (dict(tab=0), INVALID), (dict(lens=0), INVALID), (dict(new=0), INVALID), (dict(free=0), INVALID),
    (dict(used=0), INVALID), (dict(cu=0), INVALID), (dict(slot=0), INVALID), (dict(lens2=0), INVALID),
    (dict(used2=0), INVALID), (dict(R=-1), INVALID), (dict(T=-1), INVALID), (dict(F=-1), INVALID),
    (dict(M=0), INVALID), (dict(P=8), UNSUPPORTED), (dict(P=48), UNSUPPORTED), (dict(P=256), UNSUPPORTED),
    (dict(P=0), UNSUPPORTED), (dict(tab=TAB + 2), MISALIGNED), (dict(slot=SLOT + 4), MISALIGNED),
    (dict(used2=USED2 + 1), MISALIGNED),
    (dict(lens2=LEN), INVALID),         # in place: the kernel's blocks read the lengths at any time
    (dict(used2=USED), INVALID), (dict(cu=NEW + 8), INVALID), (dict(slot=TAB + 64), INVALID),
    (dict(tab=FREE + 32), INVALID), (dict(lens2=CU + 16), INVALID),
])
def test_slots_refusals(lib, kw, want):
    assert _slots(lib, **kw) == want


K, V, K8, V8, KS, VS = (0x10000000 * (i + 1) for i in range(6))


def _append(lib, k=K, v=V, k_stride=384, v_stride=384, k8=K8, v8=V8, ks=KS, vs=VS, slot=SLOT, T=20, H=3, d=128,
            blocks=10, P=32):
    return lib.fa_cache_append_e4m3(k, v, k_stride, v_stride, k8, v8, ks, vs, slot, T, H, d, blocks, P, None)


@pytest.mark.parametrize("kw,want", [
    (dict(k=0), INVALID), (dict(v=0), INVALID), (dict(k8=0), INVALID), (dict(v8=0), INVALID), (dict(ks=0), INVALID),
    (dict(vs=0), INVALID), (dict(slot=0), INVALID), (dict(T=-1), INVALID), (dict(H=0), INVALID),
    (dict(blocks=0), INVALID), (dict(d=96), UNSUPPORTED), (dict(d=0), UNSUPPORTED), (dict(P=20), UNSUPPORTED),
    (dict(H=70000, k_stride=1 << 24, v_stride=1 << 24), UNSUPPORTED), (dict(blocks=1 << 30), UNSUPPORTED),
    (dict(k_stride=376), INVALID), (dict(v_stride=0), INVALID), (dict(v_stride=-384), INVALID),
    (dict(k_stride=388), MISALIGNED), (dict(k=K + 8), MISALIGNED), (dict(v8=V8 + 8), MISALIGNED),
    (dict(ks=KS + 2), MISALIGNED), (dict(slot=SLOT + 4), MISALIGNED),
    (dict(v8=K8), INVALID), (dict(vs=KS), INVALID), (dict(k8=K), INVALID), (dict(ks=V + 256), INVALID),
    (dict(vs=SLOT), INVALID), (dict(ks=K8 + 1024), INVALID), (dict(T=0), FA_OK), (dict(T=0, k=0, slot=0), FA_OK),
])
def test_append_refusals(lib, kw, want):
    assert _append(lib, **kw) == want


Q, O, L, WS = 0x71000000, 0x72000000, 0x73000000, 0x74000000


def _fwd(lib, q=Q, stride=768, k8=K8, v8=V8, ks=KS, vs=VS, tab=0xA0000000, lens=0xA1000000, cu=0xA2000000, o=O, lse=L,
         R=4, T=9, Hq=6, H=3, d=128, blocks=10, P=32, M=5, scale=0.1, causal=1, ws=WS, n=1 << 30):
    return lib.fa_cache_fwd_e4m3(q, stride, k8, v8, ks, vs, tab, lens, cu, o, lse, R, T, Hq, H, d, blocks, P, M,
                                 scale, causal, ws, n, None)


@pytest.mark.parametrize("kw,want", [
    (dict(q=0), INVALID), (dict(k8=0), INVALID), (dict(v8=0), INVALID), (dict(ks=0), INVALID), (dict(vs=0), INVALID),
    (dict(tab=0), INVALID), (dict(lens=0), INVALID), (dict(cu=0), INVALID), (dict(o=0), INVALID),
    (dict(lse=0), INVALID), (dict(ws=0), INVALID), (dict(R=-1), INVALID), (dict(T=-1), INVALID), (dict(Hq=0), INVALID),
    (dict(Hq=7), INVALID), (dict(M=0), INVALID), (dict(causal=2), INVALID), (dict(scale=float("inf")), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(d=80), UNSUPPORTED), (dict(P=24), UNSUPPORTED),
    (dict(T=1 << 30), UNSUPPORTED), (dict(M=1 << 27), UNSUPPORTED), (dict(stride=760), INVALID),
    (dict(stride=772), MISALIGNED), (dict(q=Q + 2), MISALIGNED), (dict(o=O + 8), MISALIGNED),
    (dict(ws=WS + 8), MISALIGNED), (dict(lse=L + 2), MISALIGNED), (dict(tab=0xA0000001), MISALIGNED),
    (dict(T=0), FA_OK), (dict(R=0), FA_OK), (dict(T=0, q=0, o=0, ws=0), FA_OK),
])
def test_forward_refusals(lib, kw, want):
    assert _fwd(lib, **kw) == want


def test_forward_workspace_of_sizes_not_taken(lib):
    for bad in ((4, 9, 6, 3, 96), (0, 9, 6, 3, 128), (4, 0, 6, 3, 128), (4, 9, 7, 3, 128), (4, 9, 6, 0, 64)):
        assert lib.fa_cache_fwd_e4m3_workspace_size(*bad) == 0, bad


def test_status_string(lib):
    assert lib.fa_status_string(-6) == b"FA_ERR_INDEX"


# The Python checks run before the library is called: CPU tensors reach them.

def test_python_refuses_cpu_tensors_and_wrong_types():
    c = fa.CacheE4M3(torch.zeros(2, 1, 16, 64, dtype=torch.uint8), torch.zeros(2, 1, 16, 64, dtype=torch.uint8),
                     torch.zeros(2, 1), torch.zeros(2, 1))
    t = torch.zeros(1, 2, dtype=torch.int32)
    n = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        fa.cache_append_e4m3(torch.zeros(1, 1, 64, dtype=torch.bfloat16), torch.zeros(1, 1, 64, dtype=torch.bfloat16),
                             c, torch.zeros(1, dtype=torch.int64))
    with pytest.raises(ValueError, match="CUDA"):
        fa.cache_forward_e4m3(torch.zeros(1, 1, 64, dtype=torch.bfloat16), c, t, n, torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError, match="CUDA"):
        fa.cache_slots(t, n, n, n, n, 16, 1)
    with pytest.raises(ValueError, match="block_table"):
        fa.cache_slots(n, n, n, n, n, 16, 1)


def test_python_checks_shapes_types_and_strides():
    cpu = torch.device("cpu")
    chk, rows = cache_mod._check, cache_mod._check_rows
    x = torch.zeros(3, 4, dtype=torch.int32)
    chk("x", x, torch.int32, (3, None), cpu)
    for bad, err in ((x.long(), TypeError), (x[:, ::2], ValueError), (x[0], ValueError), ([1], TypeError),
                     (x.t().contiguous(), ValueError)):
        with pytest.raises(err):
            chk("x", bad, torch.int32, (3, None), cpu)
    q = torch.zeros(5, 8, 64, dtype=torch.bfloat16)
    rows("q", q, 8, 64, cpu)
    rows("q", q[:, 2:4], 2, 64, cpu)       # a slice of a projection
    rows("q", q[::2], 8, 64, cpu)
    rows("q", q[:0], 8, 64, cpu)
    for bad, err in ((q.float(), TypeError), (q[:, ::2], ValueError), (q.transpose(0, 1), ValueError),
                     (q[..., :32], ValueError), (q[0], ValueError), (None, TypeError)):
        with pytest.raises(err):
            rows("q", bad, None, 64, cpu)


# ------------------------------------------------------------- oracle pins

def test_oracle_slots_by_hand():
    table, cu, slots, lens, used = oracle.cache_slots([[9, -1, -1], [-1, -1, -1], [4, 5, -1]], [3, 0, 32], [2, 20, 1],
                                                      [7, 8, 1, 2], 1, 16, 25)
    assert cu == [0, 2, 22, 23] and lens == [5, 20, 33] and used == 4
    assert table == [[9, -1, -1], [8, 1, -1], [4, 5, 2]]
    assert slots[:2] == [9 * 16 + 3, 9 * 16 + 4]
    assert slots[2:22] == [8 * 16 + i for i in range(16)] + [16 + i for i in range(4)]
    assert slots[22:] == [32, -1, -1]
    # one block fewer: the third request is refused, and only it
    table, cu, slots, lens, used = oracle.cache_slots([[9, -1, -1], [-1, -1, -1], [4, 5, -1]], [3, 0, 32], [2, 20, 1],
                                                      [7, 8, 1], 1, 16, 25)
    assert cu == [0, 2, 22, 23] and lens == [5, 20, 32] and used == 3
    assert table == [[9, -1, -1], [8, 1, -1], [4, 5, -1]] and slots[22:] == [-1, -1, -1]


def test_oracle_scale_is_the_smallest_power_of_two():
    for a in (1e-25, 0.3, 1.75, 1.7578125, 447.0, 448.0, 449.0, 1e6, 3e38):
        s = oracle.block_scale(a)
        assert a <= 448 * s and a > 224 * s
    assert oracle.block_scale(0.0) == 2.0 ** -100 and oracle.block_scale(1e-37) == 2.0 ** -100


def test_oracle_growth_keeps_normal_values():
    """A block whose scale grows by 2^k keeps every value that stays normal."""
    codes, scale = np.zeros((1, 1, 16, 64), np.uint8), np.zeros((1, 1), np.float32)
    x = np.full((1, 1, 64), 1.0)
    x[0, 0, :4] = (0.5, 3.5, -1.125, 0.9375)
    oracle.cache_append(x, codes, scale, [0], 16)
    oracle.cache_append(x * 16, codes, scale, [1], 16)
    v = oracle.cache_values(codes, scale, [0], 2)
    assert np.array_equal(v[0], x[0]) and np.array_equal(v[1], 16 * x[0])


def test_oracle_attention_agrees_with_the_dense_oracle():
    """One request, as many rows as keys: causal self-attention of the values."""
    P, d, n = 16, 64, 37
    table, blocks = make_tables([n], P)
    k8, ks = make_codes(blocks, 1, P, d, 1)
    v8, vs = make_codes(blocks, 1, P, d, 2)
    q = torch.randn(n, 1, d, generator=torch.Generator().manual_seed(3)).to(torch.bfloat16)
    for causal in (False, True):
        O, L, A, S, R, W = oracle.attention_cache(q, k8, v8, ks, vs, table, [n], [0, n], 0.125, causal)
        k = torch.from_numpy(oracle.cache_values(k8.numpy(), ks.numpy(), table[0], n))
        v = torch.from_numpy(oracle.cache_values(v8.numpy(), vs.numpy(), table[0], n))
        Oref, Lref = oracle.attention_ref(q.double().transpose(0, 1)[None], k.transpose(0, 1)[None],
                                          v.transpose(0, 1)[None], 0.125, causal)
        assert torch.allclose(O[:, 0], Oref[0, 0], rtol=0, atol=1e-12)
        assert torch.allclose(L[:, 0], Lref[0, 0], rtol=0, atol=1e-12)
        assert (A >= O.abs() - 1e-12).all() and (W >= 0).all() and (R >= 0).all() and (S > 0).all()
