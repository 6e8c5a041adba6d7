"""The 8-bit key/value cache: from prompts to single tokens.

A serving step is three calls, all on the device and without a
synchronisation, so that a step can be captured into a CUDA graph:

    cu, slots, lens, used = cache_slots(table, lens, new, free, used, P, T)
    cache_append_e4m3(k, v, cache, slots)             # per layer
    o, lse = cache_forward_e4m3(q, cache, table, lens, cu, slot_map=slots)

``include/fa_fwd.h`` says what each does with every input.
"""
from __future__ import annotations

import math
from typing import NamedTuple

import torch

__all__ = ["CacheE4M3", "cache_alloc_e4m3", "cache_slots", "cache_append_e4m3", "cache_forward_e4m3",
           "cache_forward_workspace_size"]

_I32, _I64, _F32, _U8, _BF16 = torch.int32, torch.int64, torch.float32, torch.uint8, torch.bfloat16


class CacheE4M3(NamedTuple):
    """A pool of cache blocks: codes uint8 [blocks, Hkv, P, d], scales fp32
    [blocks, Hkv] in 0 .. 2^120, of K and of V."""
    k8: torch.Tensor
    v8: torch.Tensor
    k_scale: torch.Tensor
    v_scale: torch.Tensor


_empty = torch.empty
_raw_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch.cuda.current_device
_fn = None  # the library's entry points, once it is loaded


def _load():
    global _fn
    from . import load_library
    lib = load_library()
    _fn = (lib.fa_cache_slots, lib.fa_cache_append_e4m3, lib.fa_cache_fwd_e4m3_slots,
           lib.fa_cache_fwd_e4m3_workspace_size)
    return _fn


def _failed(status, where):
    from . import _raise
    _raise(status, where)


# A call on a few rows takes the GPU 3 to 15 us, so its checks are one
# expression per tensor; only where that fails is the reason looked for.

def _check(name, t, dtype, shape, device):
    """A contiguous CUDA tensor of this type; ``shape`` has None where any size will do."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    s = t.shape
    if len(s) != len(shape) or any(b is not None and a != b for a, b in zip(s, shape)):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(s)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, not on {device}")


def _check_rows(name, t, heads, d, device):
    """bf16 [T, heads, d], heads and d contiguous, any stride between tokens.
    Returns (T, heads, stride)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not _BF16:
        raise TypeError(f"{name} must be bfloat16, got {t.dtype}")
    s = t.shape
    if len(s) != 3 or (heads is not None and s[1] != heads) or s[2] != d:
        raise ValueError(f"{name} must be [T, {'heads' if heads is None else heads}, {d}], got {tuple(s)}")
    n, h, _ = s
    st = t.stride()
    if n and h and (st[2] != 1 or (h > 1 and st[1] != d)):
        raise ValueError(f"{name}: the heads of a token must be contiguous")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, not on {device}")
    return n, h, st[0] if n > 1 else h * d


def _check_cache(cache):
    k8, v8, ks, vs = cache.k8, cache.v8, cache.k_scale, cache.v_scale
    if not isinstance(k8, torch.Tensor) or k8.dim() != 4:
        raise ValueError("cache.k8 must be a uint8 [blocks, heads, block_tokens, d] tensor")
    if not k8.is_cuda:
        raise ValueError("the cache must be CUDA tensors")
    dev, shape = k8.device, k8.shape
    two = shape[:2]
    if not (k8.dtype is _U8 and k8.is_contiguous() and isinstance(v8, torch.Tensor) and v8.dtype is _U8
            and v8.shape == shape and v8.is_contiguous() and v8.device == dev and isinstance(ks, torch.Tensor)
            and ks.dtype is _F32 and ks.shape == two and ks.is_contiguous() and ks.device == dev
            and isinstance(vs, torch.Tensor) and vs.dtype is _F32 and vs.shape == two and vs.is_contiguous()
            and vs.device == dev):
        _check("cache.k8", k8, _U8, shape, dev)
        _check("cache.v8", v8, _U8, shape, dev)
        _check("cache.k_scale", ks, _F32, two, dev)
        _check("cache.v_scale", vs, _F32, two, dev)
    return dev, shape


def _ints(name, t, shape, device, dtype=_I32):
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.is_contiguous()
            and t.device == device):
        _check(name, t, dtype, shape, device)


def _call(device, stream, fn, *args):
    """``fn`` with ``device`` current and on ``stream`` (default: the current
    one), so that what it allocates belongs to that stream."""
    index = device.index
    if stream is None and index == _current_device():
        return fn(_raw_stream(index), *args)
    with torch.cuda.device(device):
        if stream is None:
            return fn(_raw_stream(index), *args)
        if isinstance(stream, int):
            stream = torch.cuda.ExternalStream(stream, device=device)
        if stream.device != device:
            raise ValueError(f"stream is on {stream.device}, the tensors on {device}")
        with torch.cuda.stream(stream):
            return fn(stream.cuda_stream, *args)


def cache_alloc_e4m3(num_blocks, heads_kv, block_tokens, d, device=None):
    """An empty cache: codes 0, scales 0 (a block gets its scale with its
    first rows)."""
    if device is None:
        device = torch.device("cuda", torch.cuda.current_device())
    shape = (num_blocks, heads_kv, block_tokens, d)
    return CacheE4M3(torch.zeros(shape, dtype=_U8, device=device), torch.zeros(shape, dtype=_U8, device=device),
                     torch.zeros(shape[:2], dtype=_F32, device=device),
                     torch.zeros(shape[:2], dtype=_F32, device=device))


def cache_slots(block_table, seq_lens, new_lens, free_blocks, free_used, block_tokens, num_tokens, stream=None):
    """Grant blocks for each request's new tokens and map them to slots.

    block_table int32 [R, max_blocks] (written in place), seq_lens and
    new_lens int32 [R], free_blocks int32 [F] with the first free_used (int32
    [1]) of them gone, num_tokens the length of the slot map.  Returns
    (cu_new int32 [R + 1], slot_map int64 [num_tokens], seq_lens_out int32
    [R], free_used_out int32 [1]).  A request that cannot be served keeps its
    length and gets slots of -1, its rows their place in cu_new; slots behind
    the last request's are -1.  Where the free blocks run out, every later
    request that needs one is refused too."""
    if not isinstance(block_table, torch.Tensor) or block_table.dim() != 2:
        raise ValueError("block_table must be an int32 [R, max_blocks] tensor")
    dev = block_table.device
    if dev.type != "cuda":
        raise ValueError("block_table must be a CUDA tensor")
    R, M = block_table.shape
    if block_table.dtype is not _I32 or not block_table.is_contiguous():
        _check("block_table", block_table, _I32, (R, M), dev)
    _ints("seq_lens", seq_lens, (R,), dev)
    _ints("new_lens", new_lens, (R,), dev)
    _ints("free_used", free_used, (1,), dev)
    if not (isinstance(free_blocks, torch.Tensor) and free_blocks.dtype is _I32 and free_blocks.dim() == 1
            and free_blocks.is_contiguous() and free_blocks.device == dev):
        _check("free_blocks", free_blocks, _I32, (None,), dev)
    if not 0 <= num_tokens <= 0x7fffffff:
        raise ValueError(f"num_tokens must be in 0 .. 2^31 - 1, got {num_tokens}")
    return _call(dev, stream, _slots, dev, block_table, seq_lens, new_lens, free_blocks, free_used, R, M, block_tokens,
                 num_tokens)


def _slots(handle, dev, table, seq_lens, new_lens, free, used, R, M, P, T):
    cu = _empty(R + 1, dtype=_I32, device=dev)
    slots = _empty(T, dtype=_I64, device=dev)
    lens = _empty(R, dtype=_I32, device=dev)
    gone = _empty(1, dtype=_I32, device=dev)
    st = (_fn or _load())[0](
        table.data_ptr(), seq_lens.data_ptr(), new_lens.data_ptr(), free.data_ptr(), used.data_ptr(), cu.data_ptr(),
        slots.data_ptr(), lens.data_ptr(), gone.data_ptr(), R, M, free.shape[0], P, T, handle)
    if st:
        _failed(st, "fa_cache_slots")
    return cu, slots, lens, gone


def cache_append_e4m3(k, v, cache, slot_map, stream=None):
    """Write new K and V rows (bf16 [T, Hkv, d], any stride between tokens)
    into the cache at the slots of ``slot_map`` (int64 [T], -1: skip), each
    run of rows in a block with the block's scale, which grows to fit."""
    dev, (blocks, H, P, d) = _check_cache(cache)
    T, _, k_stride = _check_rows("k", k, H, d, dev)
    Tv, _, v_stride = _check_rows("v", v, H, d, dev)
    if Tv != T:
        raise ValueError(f"k has {T} rows, v {Tv}")
    _ints("slot_map", slot_map, (T,), dev, _I64)
    if T:
        _call(dev, stream, _append, k, v, k_stride, v_stride, cache, slot_map, T, H, d, blocks, P)


def _append(handle, k, v, k_stride, v_stride, cache, slot_map, T, H, d, blocks, P):
    st = (_fn or _load())[1](
        k.data_ptr(), v.data_ptr(), k_stride, v_stride, cache.k8.data_ptr(), cache.v8.data_ptr(),
        cache.k_scale.data_ptr(), cache.v_scale.data_ptr(), slot_map.data_ptr(), T, H, d, blocks, P, handle)
    if st:
        _failed(st, "fa_cache_append_e4m3")


def cache_forward_workspace_size(R, T, heads, heads_kv, d) -> int:
    """Workspace bytes of ``cache_forward_e4m3`` on the current device for R
    requests and T query rows (0: none needed, or sizes it does not take)."""
    return int((_fn or _load())[3](int(R), int(T), int(heads), int(heads_kv), int(d)))


def cache_forward_e4m3(q, cache, block_table, seq_lens, cu_q, scale=None, causal=True, workspace=None, stream=None,
                       slot_map=None):
    """Attention of each request's newest tokens over its cached keys.

    q bf16 [T, Hq, d] (any stride between tokens), Hq a multiple of the
    cache's heads; request r's rows are cu_q[r] .. cu_q[r + 1] (cu_q int32
    [R + 1]), its last ones of seq_lens[r] (int32 [R]) cached tokens, whose
    blocks are block_table[r] (int32 [R, max_blocks]).  Returns (o bf16 [T,
    Hq, d], lse fp32 [T, Hq]); rows behind cu_q[R] are not written.
    ``slot_map`` (int64 [T], of cache_slots): a request that it refused, whose
    rows' slots are -1, has no keys (o 0, lse -inf); without it the rows of such
    a request are taken for the last of its older tokens.
    ``workspace`` (a CUDA tensor of cache_forward_workspace_size bytes) may be
    passed to reuse memory; calls that may overlap need one each."""
    dev, (blocks, H, P, d) = _check_cache(cache)
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
        q.data_ptr(), q_stride, cache.k8.data_ptr(), cache.v8.data_ptr(), cache.k_scale.data_ptr(),
        cache.v_scale.data_ptr(), table.data_ptr(), seq_lens.data_ptr(), cu_q.data_ptr(),
        None if slot_map is None else slot_map.data_ptr(), o.data_ptr(), lse.data_ptr(), R, T, Hq, H, d, blocks, P, M,
        scale, causal, ws.data_ptr(), ws.numel() * ws.element_size(), handle)
    if st:
        _failed(st, "fa_cache_fwd_e4m3_slots")
    return o, lse
