"""Binding of the position rotation: the frequencies of a rotary encoding, and the call that turns rows by them.

Argument marshalling only, as in block.py; cache_append_rotary there takes the same Rotary.
"""

from __future__ import annotations

import ctypes
import struct
from typing import Optional, Sequence, Union

import torch

from . import MoeW4A16Error, lib
from .block import _need, _run, _vector

MAX_ROTARY_DIM = 1024
ROTARY_NONE, ROTARY_LINEAR, ROTARY_BASE, ROTARY_TURNS, ROTARY_INDEX, ROTARY_GIVEN = range(6)
_SCALINGS = {"none": ROTARY_NONE, "linear": ROTARY_LINEAR, "base": ROTARY_BASE, "turns": ROTARY_TURNS,
             "index": ROTARY_INDEX, "given": ROTARY_GIVEN}
_BF16 = torch.bfloat16

_P, _I, _L, _D = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_double


class RotaryDesc(ctypes.Structure):
    _fields_ = [("turns", ctypes.c_void_p), ("dim", ctypes.c_int32), ("offset", ctypes.c_int32),
                ("interleaved", ctypes.c_int32), ("magnitude", ctypes.c_float)]


# a descriptor goes over as its bytes, packed once for a Rotary
_pack_desc = struct.Struct("@Piiif").pack
assert struct.calcsize("@Piiif") == ctypes.sizeof(RotaryDesc)
_SIGNATURES = {
    "rotary_frequencies": [_I, _D, _I, _D, _I, _D, _D, ctypes.POINTER(_D), ctypes.POINTER(ctypes.c_uint64)],
    "rotary": [_P, _L, _L, _P, _I, _I, _I, _P, _P, _L, _L, _P],
}
_FN = {}
for _name, _args in _SIGNATURES.items():
    _fn = getattr(lib, "moe_w4a16_" + _name)
    _fn.restype = ctypes.c_int
    _fn.argtypes = _args
    _FN[_name] = _fn


def rotary_frequencies(dim: int, theta: float = 10000.0, scaling: Union[str, int] = "none", factor: float = 1.0,
                       trained_length: int = 0, low: float = 1.0, high: float = 32.0,
                       given: Optional[Sequence[float]] = None) -> torch.Tensor:
    """The frequencies of dim / 2 pairs as the calls take them: int64 [dim / 2] on the host, each the bits of an
    unsigned number of 2^-64 turns a token. scaling: none, linear, base, turns, index (for contexts `factor` times the
    trained length; their formulas stand in moe_w4a16.h) or given (radians a token)."""
    kind = _SCALINGS.get(scaling, scaling)
    if not isinstance(kind, int):
        raise ValueError(f"scaling must be one of {', '.join(_SCALINGS)}, not {scaling!r}")
    values = None
    if given is not None:
        if kind != ROTARY_GIVEN or len(given) != dim // 2:
            raise ValueError(f"given goes with scaling='given' and has {dim // 2} elements")
        values = (_D * len(given))(*[float(f) for f in given])
    out = (ctypes.c_uint64 * max(1, dim // 2))()
    status = _FN["rotary_frequencies"](dim, theta, kind, factor, trained_length, low, high, values, out)
    if status:
        raise MoeW4A16Error(status, "rotary_frequencies")
    return torch.frombuffer(bytearray(out), dtype=torch.int64).clone()


class Rotary:
    """A rotation of positions on a device: `dim` channels of a head from `offset` on turn in pairs, dim / 2 apart or
    (interleaved) side by side; magnitude multiplies them. The other arguments are rotary_frequencies'."""

    def __init__(self, dim: int, theta: float = 10000.0, offset: int = 0, interleaved: bool = False,
                 scaling: Union[str, int] = "none", factor: float = 1.0, trained_length: int = 0, low: float = 1.0,
                 high: float = 32.0, magnitude: float = 1.0, given: Optional[Sequence[float]] = None, device=None):
        dev = torch.device(device) if device is not None else torch.device("cuda", torch.cuda.current_device())
        self.dim, self.offset, self.interleaved, self.magnitude = dim, offset, bool(interleaved), float(magnitude)
        self.turns = rotary_frequencies(dim, theta, scaling, factor, trained_length, low, high, given).to(dev)
        self._index = self.turns.get_device()
        self._desc = _pack_desc(self.turns.data_ptr(), dim, offset, int(self.interleaved), self.magnitude)

    def desc(self, index: int) -> bytes:
        """The moe_w4a16_rotary_desc for a call on CUDA device `index`."""
        if index != self._index:
            raise ValueError(f"the rotation is on {self.turns.device}, expected cuda:{index}")
        return self._desc


def rotary(x: torch.Tensor, positions: torch.Tensor, rot: Rotary, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Rows x bf16 [T, heads, dim] (any strides between tokens and heads) turned by positions int32 [T] -> out, a new
    dense tensor unless given (x itself: in place; else it does not overlap x)."""
    index = _need(x, "x", _BF16, 3).get_device()
    t, h, d = x.shape
    if out is None:
        out = torch.empty((t, h, d), dtype=_BF16, device=x.device)
    elif _need(out, "out", _BF16, 3, index).shape != x.shape:
        raise ValueError("out and x must have the same shape")
    xs, os_ = x.stride(), out.stride()
    _run("rotary", index, _FN["rotary"], x.data_ptr(), xs[0], xs[1], _vector(positions, "positions", t, index), t, h, d,
         rot.desc(index), out.data_ptr(), os_[0], os_[1])
    return out
