"""Rotary positions with several axes: aa_rope_axes_init / aa_rope_axes_apply and their autograd entry.

Tokens of images and video carry a position per axis (time, height, width); pair p of a head turns by
pos[axis of p][t] * theta_p (Eq. 6 of "When Precision Meets Position", architecture page, §3.4 "Rotary
Positional Embedding (RoPE)", with one position per axis).

    rope = RopeAxes(128, sections=(16, 24, 24), base=5e6)
    q, k = rope_axes(rope, pos, q, k)                      # pos: int32 [3, T]; differentiable in q and k
    with Plan(cu_doclens, T, Hq, Hkv, 128, rope_layout=ROPE_NONE) as plan:
        o = anchor_attention(plan, q, k, v)                # the plan does not rotate again

Like the rest of the binding this marshals arguments: the rotation is the library's kernel. Forward and backward may be
captured in a CUDA graph under PyTorch's own rule: warm up on a side stream, and keep no eager autograd graph of the same
leaves alive while capturing.
"""
from __future__ import annotations

import ctypes

from .binding import AARopeAxes, ROPE_ADJACENT, _check, lib, native

__all__ = ["RopeAxes", "rope_axes"]


class RopeAxes:
    """A multi-axis rotation: which axis and frequency each pair has. Holds no device memory; may be copied and pickled.

    sections: pairs per axis, adding up to head_dim / 2; laid one after the other, or, with interleaved=True, dealt
    to the axes in turn until each has its count. axis_of_pair gives the map itself instead. theta: [head_dim / 2]
    frequencies in place of base^(-2p/D)."""

    def __init__(self, head_dim, sections=None, base=1e4, theta=None, layout=ROPE_ADJACENT, interleaved=False,
                 axis_of_pair=None):
        head_dim = int(head_dim)
        half = head_dim // 2
        if (sections is None) == (axis_of_pair is None):
            raise ValueError("give either sections or axis_of_pair")
        if axis_of_pair is None:
            left = [int(n) for n in sections]
            if any(n < 0 for n in left) or sum(left) != half:
                raise ValueError(f"sections must be >= 0 and add up to head_dim / 2 = {half}")
            self.num_axes = len(left)
            if interleaved:
                axis_of_pair = []
                while sum(left):
                    for a, n in enumerate(left):
                        if n:
                            axis_of_pair.append(a)
                            left[a] -= 1
            else:
                axis_of_pair = [a for a, n in enumerate(left) for _ in range(n)]
        else:
            if interleaved:
                raise ValueError("interleaved goes with sections")
            axis_of_pair = [int(a) for a in axis_of_pair]
            if len(axis_of_pair) != half:
                raise ValueError(f"axis_of_pair must have head_dim / 2 = {half} entries")
            self.num_axes = max(axis_of_pair, default=0) + 1
        if theta is None:
            if not (base > 1.0 and base != float("inf")):
                raise ValueError("base must be finite and > 1")
            theta = [float(base) ** (-2.0 * p / head_dim) for p in range(half)]
        elif len(theta) != half:
            raise ValueError(f"theta must have head_dim / 2 = {half} entries")
        self.head_dim, self.layout, self.axis_of_pair = head_dim, int(layout), axis_of_pair
        self._c = AARopeAxes()
        _check(lib().aa_rope_axes_init(ctypes.addressof(self._c), head_dim, self.num_axes, self.layout,
                                       (ctypes.c_int32 * max(half, 1))(*axis_of_pair),
                                       (ctypes.c_double * max(half, 1))(*[float(x) for x in theta])))
        self._at = ctypes.addressof(self._c)

    # _at, the table's address, belongs to this object's _c: a copy or an unpickled object takes its own
    def __getstate__(self):
        return {k: v for k, v in self.__dict__.items() if k != "_at"}

    def __setstate__(self, state):
        self.__dict__.update(state)
        self._at = ctypes.addressof(self._c)

    def apply(self, pos, q, k=None, inverse=False, out_q=None, out_k=None, stream=None):
        """Rotate q [T, Hq, D] (and k [T, Hk, D]) by pos, int32 [axes, T]; inverse=True turns back. Token strides of
        slices are taken as they are; out_q = q works in place on a contiguous q."""
        r = native().rope_apply(self._at, pos, q, k, inverse, out_q, out_k, stream)
        if type(r) is int:
            _check(r)
        return r


def rope_axes(rope, pos, q, k=None):
    """RopeAxes.apply as a differentiable op: q, or (q, k), rotated. The gradient is the rotation back."""
    return native().rope_autograd(rope._at, pos, q, k)
