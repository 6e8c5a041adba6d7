"""Rotary positions: queries and keys turned by the angles of their position.

    table = rope_table(length, rot)                       # once
    q = rope(q, positions, table)                         # [T, H, d] or [B, H, N, d]
    dq = rope_backward(dq, positions, table)              # the gradient of q before it

``include/fa_fwd.h`` says what ``fa_rope`` does with every input.
"""
from __future__ import annotations

import math

import torch

from .cache import _call, _check, _failed

__all__ = ["rope_table", "rope", "rope_backward"]

_I32, _F32, _BF16 = torch.int32, torch.float32, torch.bfloat16
_empty = torch.empty
_fn = None
_usual = None  # fa_torch's, for the usual calls; None elsewhere


def _load():
    global _fn
    from . import load_library
    _fn = load_library().fa_rope
    return _fn


def _load_usual():
    global _usual
    from . import _load_torch
    _usual = _load_torch().rope
    return _usual


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


def _check_table(table, d, index):
    """(length, rot) of a table on CUDA device ``index``."""
    if not (isinstance(table, torch.Tensor) and table.dtype is _F32 and table.dim() == 3 and table.is_contiguous()
            and table.get_device() == index):
        _check("table", table, _F32, (None, None, 2), torch.device("cuda", index))
    length, half, two = table.shape
    if two != 2 or length == 0 or half == 0 or half % 8 or 2 * half > d:
        raise ValueError(f"table must be [positions, rot / 2, 2] with rot a multiple of 16 and at most d = {d}, got "
                         f"{tuple(table.shape)}")
    return length, 2 * half


def _rotate(name, x, positions, table, interleaved, out, stream, transposed):
    if not isinstance(x, torch.Tensor) or x.dtype is not _BF16:
        raise TypeError(f"{name} must be a bfloat16 tensor")
    index = x.get_device()
    if index < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    shape, st = x.shape, x.stride()
    axes = len(shape)
    if axes == 3:
        N, H, d = shape
        B, strides, usual = 1, (d, st[1], st[0]), (N,)
    elif axes == 4:
        B, H, N, d = shape
        strides, usual = st[:3], (N,)
    else:
        raise ValueError(f"{name} must be [T, H, d] or [B, H, N, d], got {tuple(shape)}")
    length, rot = _check_table(table, d, index)
    if not (isinstance(positions, torch.Tensor) and positions.dtype is _I32 and positions.is_contiguous()
            and positions.get_device() == index):
        dims = positions.dim() if isinstance(positions, torch.Tensor) else 1
        _check("positions", positions, _I32, (None,) * dims, x.device)
    per_batch = 0
    if positions.shape != usual:
        if axes == 3 or positions.shape != (B, N):
            raise ValueError(f"positions must be [{N}]{'' if axes == 3 else f' or [{B}, {N}]'}, got "
                             f"{tuple(positions.shape)}")
        per_batch = N
    if out is not None and not (isinstance(out, torch.Tensor) and out.dtype is _BF16 and out.shape == shape
                                and out.get_device() == index):
        raise ValueError(f"out must be a bfloat16 {tuple(shape)} tensor on {x.device}")
    if B * H * N == 0:
        return _empty(shape, dtype=_BF16, device=x.device) if out is None else out
    if st[-1] != 1 or (out is not None and out.stride(-1) != 1):
        raise ValueError(f"{name if st[-1] != 1 else 'out'}: the elements of a row must be contiguous")
    return _call(x.device, stream, _run, x, strides, out, axes, positions, per_batch, table, length, B, H, N, d, rot,
                 interleaved, transposed)


def _run(handle, x, strides, out, axes, positions, per_batch, table, length, B, H, N, d, rot, interleaved, transposed):
    if out is None:
        out = _empty(x.shape, dtype=_BF16, device=x.device)
        ob, oh, on = (d, d, H * d) if axes == 3 else (H * N * d, N * d, d)
    else:
        st = out.stride()
        ob, oh, on = (d, st[1], st[0]) if axes == 3 else st[:3]
    xb, xh, xn = strides
    st = (_fn or _load())(x.data_ptr(), xb, xh, xn, out.data_ptr(), ob, oh, on, positions.data_ptr(), per_batch,
                          table.data_ptr(), length, B, H, N, d, rot, bool(interleaved), transposed, handle)
    if st:
        _failed(st, "fa_rope")
    return out


def rope(x, positions, table, interleaved=False, out=None, stream=None):
    """x (bf16 [T, H, d] with positions int32 [T], or [B, H, N, d] with positions
    [N] or [B, N]; any strides but a contiguous d) with the first elements of
    each row turned by its position's angles, the table's: halves with each
    other, or (``interleaved``) neighbours.  Rows at negative positions are
    copied.  ``out`` may be x itself."""
    if out is None and stream is None:
        y = (_usual or _load_usual())(x, positions, table, interleaved, False)
        if y is not None:
            return y
    return _rotate("x", x, positions, table, interleaved, out, stream, False)


def rope_backward(dout, positions, table, interleaved=False, out=None, stream=None):
    """The gradient of rope's x, given that of its result."""
    if out is None and stream is None:
        y = (_usual or _load_usual())(dout, positions, table, interleaved, True)
        if y is not None:
            return y
    return _rotate("dout", dout, positions, table, interleaved, out, stream, True)
