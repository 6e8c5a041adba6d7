"""The 4-bit key/value cache: half the bytes of the 8-bit one, the same calls.

    cu, slots, lens, used, pos = cache_slots(table, lens, new, free, used, P, T, positions=True)
    q = rope(q, pos, angles)                                                   # per layer
    cache_append_e2m1(k, v, cache, slots, positions=pos, table=angles)         # per layer
    o, lse = cache_forward_e2m1(q, cache, table, lens, cu, slot_map=slots)     # per layer

``include/fa_fwd.h`` gives the layout and says what each does with every input.
"""
from __future__ import annotations

import math
from typing import NamedTuple

import torch

from .cache import _call, _check, _check_rows, _failed, _ints
from .rope import _check_table

__all__ = ["CacheE2M1", "cache_alloc_e2m1", "cache_append_e2m1", "cache_read_e2m1", "cache_forward_e2m1",
           "cache_forward_e2m1_workspace_size"]

_I32, _I64, _F32, _U8, _BF16 = torch.int32, torch.int64, torch.float32, torch.uint8, torch.bfloat16
_empty = torch.empty
_fn = None


def _load():
    global _fn
    from . import load_library
    lib = load_library()
    _fn = (lib.fa_cache_append_e2m1, lib.fa_cache_read_e2m1, lib.fa_cache_fwd_e2m1, lib.fa_cache_fwd_e2m1_workspace_size)
    return _fn


class CacheE2M1(NamedTuple):
    """A pool of cache blocks, uint8 [blocks, Hkv, P / 16, 18 d], and the powers of
    two (2^-64 .. 2^64) that its values are multiples of: with about the largest
    |K| / 2688 for k_unit or more nothing is cut off."""
    data: torch.Tensor
    k_unit: float = 1.0
    v_unit: float = 1.0


def _check_cache(cache):
    t = cache.data
    if not isinstance(t, torch.Tensor) or t.dim() != 4:
        raise ValueError("cache.data must be a uint8 [blocks, heads, block_tokens / 16, 18 d] tensor")
    if not t.is_cuda:
        raise ValueError("the cache must be a CUDA tensor")
    if t.dtype is not _U8 or not t.is_contiguous():
        _check("cache.data", t, _U8, t.shape, t.device)
    blocks, H, n, row = t.shape
    if row % 18:
        raise ValueError(f"cache.data: the last axis must be 18 d, got {row}")
    return t.device, blocks, H, 16 * n, row // 18


def cache_alloc_e2m1(num_blocks, heads_kv, block_tokens, d, k_unit=1.0, v_unit=1.0, device=None):
    """An empty cache (all values 0)."""
    if block_tokens not in (16, 32, 64, 128):
        raise ValueError(f"block_tokens must be 16, 32, 64 or 128, got {block_tokens}")
    if d not in (64, 128):
        raise ValueError(f"d must be 64 or 128, got {d}")
    if device is None:
        device = torch.device("cuda", torch.cuda.current_device())
    data = torch.zeros((num_blocks, heads_kv, block_tokens // 16, 18 * d), dtype=_U8, device=device)
    return CacheE2M1(data, float(k_unit), float(v_unit))


def cache_append_e2m1(k, v, cache, slot_map, positions=None, table=None, interleaved=False, stream=None):
    """Write new K and V rows (bf16 [T, Hkv, d], any stride between tokens)
    into the cache at the slots of ``slot_map`` (int64 [T], -1: skip; distinct).
    With ``positions`` (int32 [T]) and ``table`` (of rope_table) K is turned on the
    way, to the same bits as by rope before."""
    dev, blocks, H, P, d = _check_cache(cache)
    T, _, k_stride = _check_rows("k", k, H, d, dev)
    Tv, _, v_stride = _check_rows("v", v, H, d, dev)
    if Tv != T:
        raise ValueError(f"k has {T} rows, v {Tv}")
    _ints("slot_map", slot_map, (T,), dev, _I64)
    if (positions is None) != (table is None):
        raise ValueError("positions and table go together")
    length = rot = 0
    if positions is not None:
        _ints("positions", positions, (T,), dev)
        length, rot = _check_table(table, d, dev)
    if T:
        _call(dev, stream, _append, k, v, k_stride, v_stride, cache, slot_map, positions, table, length, rot,
              bool(interleaved), T, H, d, blocks, P)


def _append(handle, k, v, k_stride, v_stride, cache, slot_map, positions, table, length, rot, interleaved, T, H, d,
            blocks, P):
    st = (_fn or _load())[0](
        k.data_ptr(), v.data_ptr(), k_stride, v_stride, cache.data.data_ptr(), cache.k_unit, cache.v_unit,
        slot_map.data_ptr(), None if positions is None else positions.data_ptr(),
        None if table is None else table.data_ptr(), length, rot, interleaved, T, H, d, blocks, P, handle)
    if st:
        _failed(st, "fa_cache_append_e2m1")


def cache_read_e2m1(cache, slot_map, stream=None):
    """The cached values at the slots of ``slot_map`` (int64 [T]): K and V, bf16 [T,
    Hkv, d], exact; zeros at slots of -1."""
    dev, blocks, H, P, d = _check_cache(cache)
    if not (isinstance(slot_map, torch.Tensor) and slot_map.dtype is _I64 and slot_map.dim() == 1
            and slot_map.is_contiguous() and slot_map.device == dev):
        _check("slot_map", slot_map, _I64, (None,), dev)
    return _call(dev, stream, _read, dev, cache, slot_map, slot_map.shape[0], H, d, blocks, P)


def _read(handle, dev, cache, slot_map, T, H, d, blocks, P):
    k, v = (_empty(T, H, d, dtype=_BF16, device=dev) for _ in range(2))
    st = (_fn or _load())[1](cache.data.data_ptr(), cache.k_unit, cache.v_unit, slot_map.data_ptr(), k.data_ptr(),
                             v.data_ptr(), T, H, d, blocks, P, handle)
    if st:
        _failed(st, "fa_cache_read_e2m1")
    return k, v


def cache_forward_e2m1_workspace_size(R, T, heads, heads_kv, d) -> int:
    """Workspace bytes of ``cache_forward_e2m1`` on the current device for R
    requests and T query rows (0: none needed, or sizes it does not take)."""
    return int((_fn or _load())[3](int(R), int(T), int(heads), int(heads_kv), int(d)))


def cache_forward_e2m1(q, cache, block_table, seq_lens, cu_q, scale=None, causal=True, workspace=None, stream=None,
                       slot_map=None):
    """Attention of each request's newest tokens over its cached keys: as
    cache_forward_e4m3, over a 4-bit cache."""
    dev, blocks, H, P, d = _check_cache(cache)
    T, Hq, q_stride = _check_rows("q", q, None, d, dev)
    if Hq == 0 or H == 0 or Hq % H:
        raise ValueError(f"{Hq} query heads do not share {H} kv heads evenly")
    if not (isinstance(block_table, torch.Tensor) and block_table.dtype is _I32 and block_table.dim() == 2
            and block_table.is_contiguous() and block_table.device == dev):
        _check("block_table", block_table, _I32, (None, None), dev)
    R, M = block_table.shape
    _ints("seq_lens", seq_lens, (R,), dev)
    _ints("cu_q", cu_q, (R + 1,), dev)
    if slot_map is not None:
        _ints("slot_map", slot_map, (T,), dev, _I64)
    if workspace is not None and (workspace.device != dev or not workspace.is_contiguous()):
        raise ValueError(f"workspace must be a contiguous tensor on {dev}")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    return _call(dev, stream, _forward, dev, q, q_stride, cache, block_table, seq_lens, cu_q, slot_map, float(scale),
                 bool(causal), workspace, R, T, Hq, H, d, blocks, P, M)


def _forward(handle, dev, q, q_stride, cache, table, seq_lens, cu_q, slot_map, scale, causal, ws, R, T, Hq, H, d, blocks,
             P, M):
    o = _empty(T, Hq, d, dtype=_BF16, device=dev)
    lse = _empty(T, Hq, dtype=_F32, device=dev)
    fn = _fn or _load()
    if ws is None:
        ws = _empty(fn[3](R, T, Hq, H, d), dtype=_U8, device=dev)
    st = fn[2](
        q.data_ptr(), q_stride, cache.data.data_ptr(), cache.k_unit, cache.v_unit, table.data_ptr(),
        seq_lens.data_ptr(), cu_q.data_ptr(), None if slot_map is None else slot_map.data_ptr(), o.data_ptr(),
        lse.data_ptr(), R, T, Hq, H, d, blocks, P, M, scale, causal, ws.data_ptr(), ws.numel() * ws.element_size(), handle)
    if st:
        _failed(st, "fa_cache_fwd_e2m1")
    return o, lse
