"""Rotary positions (include/qsa.h, "Rotary positions").  Argument marshalling only.

    rope = Rope(128, base=1e6, scaling=RopeScaling("parts", 32.0, original_tokens=8192))
    rotate(rope, positions, q, out)                    # rows by themselves
    paged_append(cache, batch, k, v, rope=rope, q=q, q_out=out)   # on their way into a cache
"""
from __future__ import annotations

import ctypes
import dataclasses
from typing import Sequence

import torch

from . import BF16, F32, _check, _dtype_code, lib
from .calls import _call_at

MAX_ROPE_PAIRS = 128
_SCALINGS = {None: 0, "linear": 1, "parts": 2}


class RopeDesc(ctypes.Structure):
    _fields_ = [("rot_dim", ctypes.c_int32), ("pairs", ctypes.c_int32), ("magnitude", ctypes.c_float),
                ("reserved", ctypes.c_int32), ("turns", ctypes.c_uint64 * MAX_ROPE_PAIRS)]


def declare(L: ctypes.CDLL):
    """Argument types of the entry points, on the loaded library."""
    vp, i32, i64, f64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_double
    ropep = ctypes.POINTER(RopeDesc)
    L.qsa_rope_frequencies.argtypes = [i32, f64, i32, f64, f64, f64, f64, ctypes.POINTER(f64), ctypes.POINTER(ctypes.c_float)]
    L.qsa_rope_init.argtypes = [ropep, i32, i32, ctypes.POINTER(f64), ctypes.c_float]
    L.qsa_rotate.argtypes = [ropep, vp, i32, i32, i32, i32, vp, i64, i64, vp, i64, i64, vp]
    for name in ("qsa_rope_frequencies", "qsa_rope_init", "qsa_rotate"):
        getattr(L, name).restype = i32


@dataclasses.dataclass(frozen=True)
class RopeScaling:
    """How frequencies are stretched for contexts `factor` times as long: "linear"
    (all of them), or "parts": those that turn more than `fast` times over
    original_tokens stay, those that turn less than `slow` times are divided, with a
    ramp between the two that is linear in how often a pair turns.  Models trained with
    a ramp that is linear in the pair's index take Rope(frequencies=) instead
    (include/qsa.h has both formulas)."""
    kind: str
    factor: float
    original_tokens: float = 0.0
    fast: float = 32.0
    slow: float = 1.0


class Rope:
    """A rotation of the first rot_dim channels of a head: channels (i, i + rot_dim / 2),
    or with pairs=True neighbours (2i, 2i + 1).  Its frequencies (radians a position)
    are base^(-2i / rot_dim), scaled as asked, or the given ones; magnitude is the
    factor on what is rotated (default: the scaling's own, or 1)."""

    def __init__(self, rot_dim: int, *, base: float = 10000.0, pairs: bool = False, scaling: RopeScaling | None = None,
                 frequencies: Sequence[float] | None = None, magnitude: float | None = None):
        n = max(int(rot_dim) // 2, 1)
        w = (ctypes.c_double * n)()
        own = ctypes.c_float(1.0)
        if frequencies is not None:
            if scaling is not None:
                raise ValueError("given frequencies are not scaled")
            if len(frequencies) != int(rot_dim) // 2:
                raise ValueError(f"rot_dim {rot_dim} takes {int(rot_dim) // 2} frequencies, not {len(frequencies)}")
            w[:] = [float(x) for x in frequencies]
        else:
            s = scaling or RopeScaling(None, 1.0)
            if s.kind not in _SCALINGS:
                raise ValueError(f"unknown scaling {s.kind!r}")
            _check("qsa_rope_frequencies", lib().qsa_rope_frequencies(
                int(rot_dim), float(base), _SCALINGS[s.kind], float(s.factor), float(s.original_tokens), float(s.fast),
                float(s.slow), w, ctypes.byref(own)))
        self.desc = RopeDesc()
        _check("qsa_rope_init", lib().qsa_rope_init(ctypes.byref(self.desc), int(rot_dim), int(bool(pairs)), w,
                                                    own.value if magnitude is None else float(magnitude)))
        self.rot_dim, self.pairs, self.magnitude = int(rot_dim), bool(pairs), float(self.desc.magnitude)
        self.frequencies = tuple(w[:self.rot_dim // 2])
        self.byref = ctypes.byref(self.desc)


_KINDS = {torch.float32: F32, torch.bfloat16: BF16}


def _strides(shape, strides):
    """Row and head strides of [rows, heads, dim]; those of an axis of one do not matter."""
    return strides[0] if shape[0] > 1 else shape[1] * shape[2], strides[1] if shape[1] > 1 else shape[2]


def rotate(rope: Rope, positions: torch.Tensor, x: torch.Tensor, out: torch.Tensor | None = None, stream=None):
    """out[r, h] = x[r, h] rotated for position positions[r] (int32, on the GPU).  x is
    [rows, heads, dim] of f32 or bf16 with unit channel stride; out may be x itself, and
    is x by default."""
    shape, x_strides, device, dtype = x.shape, x.stride(), x.get_device(), x.dtype
    if out is None or out is x:
        out, out_strides = x, x_strides
    else:
        out_strides = out.stride()
        if out.shape != shape or out.dtype is not dtype or out.get_device() != device or (
                device < 0 and out.device != x.device):   # (what is no GPU has -1 in common)
            raise ValueError("x and out must be [rows, heads, dim] of one shape, dtype and device")
    if len(shape) != 3:
        raise ValueError("x and out must be [rows, heads, dim] of one shape, dtype and device")
    kind = _KINDS.get(dtype)
    if kind is None:
        raise TypeError(f"x must be float32 or bfloat16, not {dtype}")
    rows, heads, dim = shape
    if (x_strides[2] != 1 or out_strides[2] != 1) and dim > 1:
        raise ValueError("x and out need unit channel stride")
    if positions.dtype is not torch.int32 or positions.shape != (rows,) or not positions.is_contiguous():
        raise TypeError("positions must be a contiguous int32 vector with an entry for each row")
    if positions.get_device() != device or (device < 0 and positions.device != x.device):
        raise ValueError(f"positions is on {positions.device}, x on {x.device}")
    if rows > 1 and heads > 1:
        x_row, x_head, _ = x_strides
        y_row, y_head, _ = out_strides
    else:
        x_row, x_head = _strides(shape, x_strides)
        y_row, y_head = _strides(shape, out_strides)
    _call_at("qsa_rotate", device, stream, rope.byref, positions.data_ptr(), rows, heads, dim, kind, x.data_ptr(), x_row,
          x_head, out.data_ptr(), y_row, y_head)
    return out
