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

import contextlib
import ctypes

import torch

from .binding import AARopeAxes, ROPE_ADJACENT, _check, _stream_ptr, lib

__all__ = ["RopeAxes", "RopeAxesFn", "rope_axes"]


# The single-token calls take a few microseconds on the GPU, so their host side is kept lean: plain attribute tests, no
# context managers or temporary objects on the common path.
_NOTHING = contextlib.nullcontext()


def _on(stream):
    """Allocate on the stream that the kernels will run on."""
    return _NOTHING if stream is None else torch.cuda.stream(stream)


def _check_rows(name, x, T, H, D, device):
    """x is a bf16 tensor [T, H, D] on `device` (T, H None: any)."""
    if not isinstance(x, torch.Tensor) or x.dtype is not torch.bfloat16 or x.device != device:
        raise ValueError(f"{name} must be a bfloat16 tensor on {device}")
    shape = x.shape
    if len(shape) != 3 or shape[2] != D or (T is not None and shape[0] != T) or (H is not None and shape[1] != H):
        want = tuple("any" if n is None else n for n in (T, H, D))
        raise ValueError(f"{name} must have shape {want}, got {tuple(shape)}")


def _check_tensor(name, x, shape, dtype, device):
    """x is a contiguous tensor of `dtype` and `shape` on `device`."""
    if not isinstance(x, torch.Tensor) or x.dtype is not dtype or x.device != device:
        raise ValueError(f"{name} must be a {dtype} tensor on {device}")
    if x.shape != shape or not x.is_contiguous():
        raise ValueError(f"{name} must be contiguous with shape {tuple(shape)}, got {tuple(x.shape)}")


def _rows(x):
    """(x, token stride) as the kernels read it: a token's heads contiguous, 16-byte aligned rows; copied if it is not."""
    T, H, D = x.shape
    a, b, c = x.stride()
    if c == 1 and (b == D or H == 1) and x.data_ptr() % 16 == 0:
        if T <= 1:
            return x, H * D
        if a >= H * D and a % 8 == 0:
            return x, a
    x = x.contiguous()
    return (x if x.data_ptr() % 16 == 0 else x.clone()), H * D


def _out(name, out, like):
    """The caller's output tensor, checked, or a new contiguous one of the shape of `like`."""
    if out is None:
        return torch.empty(like.shape, dtype=like.dtype, device=like.device)
    _check_tensor(name, out, like.shape, like.dtype, like.device)
    return out


class RopeAxes:
    """A multi-axis rotation: which axis and frequency each pair has. Holds no device memory.

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

    def _positions(self, pos, T, device):
        if not isinstance(pos, torch.Tensor) or pos.dtype is not torch.int32 or pos.device != device:
            raise ValueError(f"pos must be an int32 tensor on {device}")
        shape = pos.shape
        if shape != (self.num_axes, T) and not (self.num_axes == 1 and shape == (T,)):
            raise ValueError(f"pos must have shape ({self.num_axes}, {T}), got {tuple(shape)}")
        return pos.contiguous()

    def apply(self, pos, q, k=None, inverse=False, out_q=None, out_k=None, stream=None):
        """Rotate q [T, Hq, D] (and k [T, Hk, D]) by pos, int32 [axes, T]; inverse=True turns back. Token strides of
        slices are taken as they are; out_q = q works in place on a contiguous q."""
        if not isinstance(q, torch.Tensor) or not q.is_cuda:
            raise ValueError("q must be a CUDA tensor")
        dev = q.device
        index = dev.index
        _check_rows("q", q, None, None, self.head_dim, dev)
        if index != torch.cuda.current_device():
            raise ValueError(f"q is on {dev}, which is not the current device")
        T, hq, _ = q.shape
        if k is not None:
            _check_rows("k", k, T, None, self.head_dim, dev)
        elif out_k is not None:
            raise ValueError("out_k goes with k")
        with _on(stream):
            pos = self._positions(pos, T, dev)
            yq = _out("out_q", out_q, q)
            q, sq = _rows(q)
            yk, kp, sk, yp, hk = None, None, 0, None, 0
            if k is not None:
                yk = _out("out_k", out_k, k)
                k, sk = _rows(k)
                kp, yp, hk = k.data_ptr(), yk.data_ptr(), k.shape[1]
            status = lib().aa_rope_axes_apply(self._at, pos.data_ptr(), T, q.data_ptr(), sq, yq.data_ptr(), hq, kp, sk, yp, hk,
                                              1 if inverse else 0, _stream_ptr(stream, index))
            if status:
                _check(status)
        return yq if k is None else (yq, yk)


class RopeAxesFn(torch.autograd.Function):
    """The rotation is orthogonal: its gradient is the rotation back."""

    @staticmethod
    def forward(ctx, rope, pos, inverse, q, k):
        ctx.rope, ctx.inverse = rope, inverse
        ctx.save_for_backward(pos)
        out = rope.apply(pos, q, k, inverse=inverse)
        return (out, None) if k is None else out

    @staticmethod
    def backward(ctx, gq, gk):
        (pos,) = ctx.saved_tensors
        need_q, need_k = ctx.needs_input_grad[3:]
        if need_q:
            gq, gk = RopeAxesFn.apply(ctx.rope, pos, not ctx.inverse, gq, gk if need_k else None)
        elif need_k:
            gq, gk = None, RopeAxesFn.apply(ctx.rope, pos, not ctx.inverse, gk, None)[0]
        return None, None, None, gq if need_q else None, gk if need_k else None


def rope_axes(rope, pos, q, k=None):
    """RopeAxes.apply as a differentiable op: q, or (q, k), rotated."""
    yq, yk = RopeAxesFn.apply(rope, pos, False, q, k)
    return yq if k is None else (yq, yk)
