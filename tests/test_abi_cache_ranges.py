"""Refusals of the cache forward's entry point with a slot map, on the host:
fake addresses that are never dereferenced."""
import pytest

import exact_attention_forward_04_gb300 as fa

FA_OK, INVALID, MISALIGNED = 0, -1, -3
Q, K8, V8, KS, VS, TAB, LEN, CU, SLOT, O, L, WS = (0x10000000 * (i + 1) for i in range(12))


@pytest.fixture(scope="module")
def lib():
    from exact_attention_forward_04_gb300 import _build
    _build.build()
    return fa.load_library()


@pytest.mark.parametrize("kw,want", [
    (dict(slot=SLOT + 4), MISALIGNED), (dict(q=0), INVALID), (dict(R=-1), INVALID), (dict(ws=WS + 8), MISALIGNED),
    (dict(T=0), FA_OK), (dict(R=0, slot=SLOT + 1), FA_OK),
])
def test_refusals_with_a_slot_map(lib, kw, want):
    a = dict(dict(q=Q, slot=SLOT, R=4, T=9, ws=WS), **kw)
    assert lib.fa_cache_fwd_e4m3_slots(a["q"], 768, K8, V8, KS, VS, TAB, LEN, CU, a["slot"], O, L, a["R"], a["T"], 6, 3,
                                       128, 10, 32, 5, 0.1, 1, a["ws"], 1 << 30, None) == want
