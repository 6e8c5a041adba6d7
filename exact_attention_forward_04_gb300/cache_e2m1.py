"""The 4-bit key/value cache: 9/16 of the bytes of the 8-bit one, the same calls.

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

from .cache import _call, _check, _check_rows, _failed
from .rope import _check_table

__all__ = ["CacheE2M1", "cache_alloc_e2m1", "cache_append_e2m1", "cache_read_e2m1", "cache_forward_e2m1",
           "cache_forward_e2m1_workspace_size"]

_I32, _I64, _F32, _U8, _BF16 = torch.int32, torch.int64, torch.float32, torch.uint8, torch.bfloat16
_empty = torch.empty
_fn = None
_usual = None  # fa_torch, for the usual calls: None is its answer to others


def _load_usual():
    global _usual
    from . import _load_torch
    _usual = _load_torch()
    return _usual


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


def _check_cache(t):
    """(CUDA device index, blocks, heads, block_tokens, d) of a cache's array."""
    if not isinstance(t, torch.Tensor) or t.dim() != 4:
        raise ValueError("cache.data must be a uint8 [blocks, heads, block_tokens / 16, 18 d] tensor")
    index = t.get_device()
    if index < 0:
        raise ValueError("the cache must be a CUDA tensor")
    if t.dtype is not _U8 or not t.is_contiguous():
        _check("cache.data", t, _U8, t.shape, t.device)
    blocks, H, n, row = t.shape
    if row % 18:
        raise ValueError(f"cache.data: the last axis must be 18 d, got {row}")
    return index, blocks, H, 16 * n, row // 18


def _rows(name, t, heads, d, index):
    """(T, elements between tokens) of bf16 [T, heads, d] rows."""
    n, _, stride = _check_rows(name, t, heads, d, torch.device("cuda", index))
    return n, stride


def _vector(name, t, dtype, n, index):
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == (n,) and t.is_contiguous()
            and t.get_device() == index):
        _check(name, t, dtype, (n,), torch.device("cuda", index))


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
    data, k_unit, v_unit = cache
    if stream is None and (_usual or _load_usual()).append(k, v, data, k_unit, v_unit, slot_map, positions, table,
                                                           interleaved):
        return
    index, blocks, H, P, d = _check_cache(data)
    T, k_stride = _rows("k", k, H, d, index)
    Tv, v_stride = _rows("v", v, H, d, index)
    if Tv != T:
        raise ValueError(f"k has {T} rows, v {Tv}")
    _vector("slot_map", slot_map, _I64, T, index)
    angles = where = None
    length = rot = 0
    if positions is not None and table is not None:
        _vector("positions", positions, _I32, T, index)
        length, rot = _check_table(table, d, index)
        angles, where = table.data_ptr(), positions.data_ptr()
    elif positions is not None or table is not None:
        raise ValueError("positions and table go together")
    if T:
        _call(data.device, stream, _append, k.data_ptr(), v.data_ptr(), k_stride, v_stride, data.data_ptr(), k_unit,
              v_unit, slot_map.data_ptr(), where, angles, length, rot, bool(interleaved), T, H, d, blocks, P)


def _append(handle, *args):
    st = (_fn or _load())[0](*args, handle)
    if st:
        _failed(st, "fa_cache_append_e2m1")


def cache_read_e2m1(cache, slot_map, stream=None):
    """The cached values at the slots of ``slot_map`` (int64 [T]): K and V, bf16 [T,
    Hkv, d], exact; zeros at slots of -1."""
    data, k_unit, v_unit = cache
    if stream is None:
        kv = (_usual or _load_usual()).read(data, k_unit, v_unit, slot_map)
        if kv is not None:
            return kv
    index, blocks, H, P, d = _check_cache(data)
    if not (isinstance(slot_map, torch.Tensor) and slot_map.dtype is _I64 and slot_map.dim() == 1
            and slot_map.is_contiguous() and slot_map.get_device() == index):
        _check("slot_map", slot_map, _I64, (None,), data.device)
    dev = data.device
    return _call(dev, stream, _read, dev, data, k_unit, v_unit, slot_map, slot_map.shape[0], H, d, blocks, P)


def _read(handle, dev, data, k_unit, v_unit, slot_map, T, H, d, blocks, P):
    k = _empty((T, H, d), dtype=_BF16, device=dev)
    v = _empty((T, H, d), dtype=_BF16, device=dev)
    st = (_fn or _load())[1](data.data_ptr(), k_unit, v_unit, slot_map.data_ptr(), k.data_ptr(), v.data_ptr(), T, H, d,
                             blocks, P, handle)
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
    data, k_unit, v_unit = cache
    if stream is None:
        out = (_usual or _load_usual()).forward(q, data, k_unit, v_unit, block_table, seq_lens, cu_q, scale, causal,
                                                workspace, slot_map)
        if out is not None:
            return out
    index, blocks, H, P, d = _check_cache(data)
    dev = data.device
    if not isinstance(q, torch.Tensor) or q.dim() != 3:
        _check_rows("q", q, None, d, dev)
    Hq = q.shape[1]
    T, q_stride = _rows("q", q, Hq, d, index)
    if Hq == 0 or H == 0 or Hq % H:
        raise ValueError(f"{Hq} query heads do not share {H} kv heads evenly")
    if not (isinstance(block_table, torch.Tensor) and block_table.dtype is _I32 and block_table.dim() == 2
            and block_table.is_contiguous() and block_table.get_device() == index):
        _check("block_table", block_table, _I32, (None, None), dev)
    R, M = block_table.shape
    _vector("seq_lens", seq_lens, _I32, R, index)
    _vector("cu_q", cu_q, _I32, R + 1, index)
    if slot_map is not None:
        _vector("slot_map", slot_map, _I64, T, index)
        slot_map = slot_map.data_ptr()
    if workspace is not None and (workspace.get_device() != index or not workspace.is_contiguous()):
        raise ValueError(f"workspace must be a contiguous tensor on {dev}")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    return _call(dev, stream, _forward, dev, q.data_ptr(), q_stride, data.data_ptr(), k_unit, v_unit,
                 block_table.data_ptr(), seq_lens.data_ptr(), cu_q.data_ptr(), slot_map, scale, bool(causal), workspace,
                 (R, T, Hq, H, d), blocks, P, M)


def _forward(handle, dev, q, q_stride, data, k_unit, v_unit, table, seq_lens, cu_q, slot_map, scale, causal, ws, sizes,
             blocks, P, M):
    R, T, Hq, H, d = sizes
    o = _empty((T, Hq, d), dtype=_BF16, device=dev)
    lse = _empty((T, Hq), dtype=_F32, device=dev)
    if ws is None:
        ws = _empty((_fn or _load())[3](*sizes), dtype=_U8, device=dev)
    st = (_fn or _load())[2](q, q_stride, data, k_unit, v_unit, table, seq_lens, cu_q, slot_map, o.data_ptr(),
                             lse.data_ptr(), R, T, Hq, H, d, blocks, P, M, scale, causal, ws.data_ptr(),
                             ws.numel() * ws.element_size(), handle)
    if st:
        _failed(st, "fa_cache_fwd_e2m1")
    return o, lse
