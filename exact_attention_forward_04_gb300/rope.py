"""Rotary positions: queries and keys turned by the angles of their position.

    table = rope_table(length, rot)                       # once
    q = rope(q, positions, table)                         # [T, H, d] or [B, H, N, d]
    dq = rope_backward(dq, positions, table)              # the gradient of q before it

``include/fa_fwd.h`` says what ``fa_rope`` does with every input.
"""
from __future__ import annotations

import ctypes
import math

import torch

from .cache import _call, _check, _failed

__all__ = ["rope_table", "rope", "rope_backward"]

_I32, _F32, _BF16 = torch.int32, torch.float32, torch.bfloat16
_Strides = ctypes.c_longlong * 3
_fn = None


def _load():
    global _fn
    from . import load_library
    _fn = load_library().fa_rope
    return _fn


def rope_table(length, rot, base=10000.0, factor=1.0, original_length=None, low=1.0, high=32.0, magnitude=1.0,
               device=None):
    """(cos, sin) of positions 0 .. length - 1 and frequencies base^(-2 i / rot):
    fp32 [length, rot / 2, 2], from 64-bit angles.

    ``factor`` stretches positions for contexts longer than the trained one: all
    frequencies are divided by it or, with ``original_length``, by how often one
    turns over that length: more than ``high`` times, and it is kept; less than
    ``low`` times, and it is divided; in between the two are mixed linearly
    (interpolation by parts, as in "YaRN: Efficient Context Window Extension of
    Large Language Models").  ``magnitude`` multiplies all entries (that paper:
    0.1 ln(factor) + 1)."""
    if rot <= 0 or rot % 16:
        raise ValueError(f"rot must be a positive multiple of 16, got {rot}")
    if length <= 0:
        raise ValueError(f"length must be positive, got {length}")
    if not (base > 0 and factor > 0 and math.isfinite(base) and math.isfinite(factor)):
        raise ValueError("base and factor must be positive and finite")
    if device is None:
        device = torch.device("cuda", torch.cuda.current_device())
    f = base ** (-torch.arange(rot // 2, dtype=torch.float64) * 2 / rot)
    if original_length is None:
        f = f / factor
    else:
        if not high > low:
            raise ValueError(f"high must be above low, got {high} and {low}")
        keep = ((original_length * f / (2 * math.pi) - low) / (high - low)).clamp(0, 1)
        f = f * keep + f / factor * (1 - keep)
    angle = torch.arange(length, dtype=torch.float64)[:, None] * f
    return torch.stack((angle.cos(), angle.sin()), -1).mul_(magnitude).to(_F32).to(device)


def _check_table(table, d, device):
    if not (isinstance(table, torch.Tensor) and table.dtype is _F32 and table.dim() == 3 and table.shape[2] == 2
            and table.is_contiguous() and table.device == device):
        _check("table", table, _F32, (None, None, 2), device)
    rot = 2 * table.shape[1]
    if rot == 0 or rot % 16 or rot > d:
        raise ValueError(f"table: {rot} elements to turn must be a multiple of 16 and at most d = {d}")
    if table.shape[0] == 0:
        raise ValueError("table has no positions")
    return table.shape[0], rot


def _rotate(name, x, positions, table, interleaved, out, stream, transposed):
    if not isinstance(x, torch.Tensor) or x.dtype is not _BF16:
        raise TypeError(f"{name} must be a bfloat16 tensor")
    if not x.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    dev, shape = x.device, x.shape
    if len(shape) not in (3, 4):
        raise ValueError(f"{name} must be [T, H, d] or [B, H, N, d], got {tuple(shape)}")
    d = shape[-1]
    length, rot = _check_table(table, d, dev)
    if not (isinstance(positions, torch.Tensor) and positions.dtype is _I32 and positions.is_contiguous()
            and positions.device == dev):
        _check("positions", positions, _I32, (None,) * (positions.dim() if isinstance(positions, torch.Tensor) else 1),
               dev)
    if len(shape) == 3:
        B, N, H = 1, shape[0], shape[1]
        if positions.shape != (N,):
            raise ValueError(f"positions must be [{N}], got {tuple(positions.shape)}")
        axes, per_batch = (None, 1, 0), 0
    else:
        B, H, N = shape[0], shape[1], shape[2]
        if positions.shape != (N,) and positions.shape != (B, N):
            raise ValueError(f"positions must be [{N}] or [{B}, {N}], got {tuple(positions.shape)}")
        axes, per_batch = (0, 1, 2), N if positions.dim() == 2 else 0
    if out is not None:
        if not (isinstance(out, torch.Tensor) and out.dtype is _BF16 and out.shape == shape and out.device == dev):
            raise ValueError(f"out must be a bfloat16 {tuple(shape)} tensor on {dev}")
    if H == 0 or B == 0 or N == 0:
        return torch.empty(shape, dtype=_BF16, device=dev) if out is None else out
    for what, t in ((name, x), ("out", out)):
        if t is not None and t.stride(-1) != 1:
            raise ValueError(f"{what}: the elements of a row must be contiguous")
    return _call(dev, stream, _run, dev, x, out, axes, positions, per_batch, table, length, B, H, N, d, rot,
                 bool(interleaved), transposed)


def _strides(t, axes, sizes, d):
    """Of batches, heads and tokens; an axis of one element gets d."""
    st = t.stride()
    return _Strides(*(d if n == 1 or i is None else st[i] for i, n in zip(axes, sizes)))


def _run(handle, dev, x, out, axes, positions, per_batch, table, length, B, H, N, d, rot, interleaved, transposed):
    if out is None:
        out = torch.empty(x.shape, dtype=_BF16, device=dev)
    sizes = (B, H, N)
    st = (_fn or _load())(
        x.data_ptr(), _strides(x, axes, sizes, d), out.data_ptr(), _strides(out, axes, sizes, d),
        positions.data_ptr(), per_batch, table.data_ptr(), length, B, H, N, d, rot, interleaved, transposed, handle)
    if st:
        _failed(st, "fa_rope")
    return out


def rope(x, positions, table, interleaved=False, out=None, stream=None):
    """x (bf16 [T, H, d] with positions int32 [T], or [B, H, N, d] with positions
    [N] or [B, N]; any strides but a contiguous d) with the first elements of
    each row turned by its position's angles, the table's: halves with each
    other, or (``interleaved``) neighbours.  Rows at negative positions are
    copied.  ``out`` may be x itself."""
    return _rotate("x", x, positions, table, interleaved, out, stream, False)


def rope_backward(dout, positions, table, interleaved=False, out=None, stream=None):
    """The gradient of rope's x, given that of its result."""
    return _rotate("dout", dout, positions, table, interleaved, out, stream, True)
