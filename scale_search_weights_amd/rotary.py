"""Rotary positions: Python binding of ``include/nvfp4_rotary.h``.

A ``Rotary`` says how a head's channels turn: a frequency of each pair of channels, and the axis of
the token's position that drives it (one axis for text; time, height and width for images and
video). ``rotate`` turns queries and keys, with gradients; ``kvcache.append`` turns new keys on
their way into the cache by the same rule.

    rot = rotary.Rotary.create(128, base=1e6)                       # text
    rot = rotary.Rotary.create(128, base=1e6, sections=(16, 24, 24))  # time, height, width
    q = rotary.rotate(q, positions, rot)                            # positions [tokens] or [axes, tokens]

As in ``nvfp4``, this module checks and marshals arguments; the work is done by the HIP kernels on
the current stream, and there is no CPU fallback.
"""
from __future__ import annotations

import ctypes
import math

import torch
from torch.autograd.forward_ad import unpack_dual

from . import nvfp4
from .nvfp4 import _I, _I64, _P, _check, _dt, _Fixed, _need

MAX_HEAD_DIM = 1024
MAX_PAIRS = 512
MAX_AXES = 16


class _Rotary(ctypes.Structure):
    _fields_ = [("inv_freq", _P), ("axis", _P), ("pairs", _I64), ("axes", _I64), ("factor", ctypes.c_double),
                ("adjacent", _I)]


_SIGS = {
    "nvfp4_rotate": (_I, [_P, _P, _I64, _P, _I, _I64, _I64, _I64, _I64, _I64, _P, _I64, _I64, _I, _P]),
}
_bound = None


def lib():
    """libnvfp4 with the rotation bound (raises if it was not built)."""
    global _bound
    if _bound is None:
        L = nvfp4.lib()
        for name, (res, args) in _SIGS.items():
            f = getattr(L, name)
            f.restype, f.argtypes = res, args
        _bound = L
    return _bound


class Rotary(_Fixed):
    """How a head's first 2 * pairs channels turn; the others pass through.

    inv_freq [pairs] (fp64, on the GPU): pair i turns by position * inv_freq[i]; pairs is a multiple of
    4 (of 8 for ``kvcache.append``). axis [pairs] (int32, same GPU): the row of the positions that
    drives the pair, in any order; None: all on axis 0. A pair is channels i and i + pairs, or 2 i and
    2 i + 1 with ``adjacent``. Cosines and sines are multiplied by ``factor``. The tensors may be
    changed between calls; an attribute cannot be replaced."""

    def __init__(self, inv_freq: torch.Tensor, axis: torch.Tensor | None = None, *, axes: int = 1,
                 adjacent: bool = False, factor: float = 1.0):
        _need(inv_freq, "inv_freq")
        if inv_freq.dtype != torch.float64 or inv_freq.dim() != 1:
            raise TypeError("inv_freq must be torch.float64 with 1 dimension")
        if inv_freq.requires_grad:
            raise ValueError("no gradient flows to inv_freq")
        pairs = inv_freq.shape[0]
        if pairs < 4 or pairs % 4 or pairs > MAX_PAIRS:
            raise ValueError(f"the pairs must be a multiple of 4 up to {MAX_PAIRS}, got {pairs}")
        if not 1 <= axes <= MAX_AXES:
            raise ValueError(f"axes must be 1 to {MAX_AXES}, got {axes}")
        if axis is not None:
            _need(axis, "axis")
            if axis.device != inv_freq.device:
                raise ValueError(f"axis is on {axis.device}, expected {inv_freq.device}")
            if axis.dtype != torch.int32 or axis.shape != (pairs,):
                raise TypeError(f"axis must be torch.int32 [{pairs}]")
        elif axes != 1:
            raise ValueError("several axes need the axis of each pair")
        if not math.isfinite(factor):
            raise ValueError(f"factor must be finite, got {factor}")
        self.inv_freq, self.axis, self.pairs, self.axes = inv_freq, axis, pairs, axes
        self.adjacent, self.factor, self.device = bool(adjacent), float(factor), inv_freq.device
        self._index = self.device.index
        self._c = _Rotary(inv_freq.data_ptr(), None if axis is None else axis.data_ptr(), pairs, axes,
                          self.factor, int(self.adjacent))
        self._ref = ctypes.addressof(self._c)

    def _of(self, inv_freq: torch.Tensor, axis: torch.Tensor | None) -> "Rotary":
        """The Rotary with this one's tensors or copies of them."""
        if inv_freq.data_ptr() == self._c.inv_freq and (axis is None or axis.data_ptr() == self._c.axis):
            return self
        return Rotary(inv_freq, axis, axes=self.axes, adjacent=self.adjacent, factor=self.factor)

    @classmethod
    def create(cls, rotary_dim: int, base: float = 10000.0, sections=None, *, adjacent: bool = False,
               factor: float = 1.0, device="cuda") -> "Rotary":
        """Frequencies base ** (-i / pairs) of rotary_dim / 2 pairs. sections: how many pairs in a row
        belong to each axis (their sum is the number of pairs)."""
        if rotary_dim < 8 or rotary_dim % 8:
            raise ValueError(f"rotary_dim must be a multiple of 8, got {rotary_dim}")
        pairs = rotary_dim // 2
        axis, axes = None, 1
        if sections is not None:
            sections = [int(n) for n in sections]
            if min(sections, default=-1) < 0 or sum(sections) != pairs:
                raise ValueError(f"the sections must add up to {pairs} pairs, got {sections}")
            axes = len(sections)
            axis = torch.cat([torch.full((n,), a, dtype=torch.int32) for a, n in enumerate(sections)]).to(device)
        inv_freq = float(base) ** (-torch.arange(pairs, dtype=torch.float64) / pairs)
        return cls(inv_freq.to(device), axis, axes=axes, adjacent=adjacent, factor=factor)


def _stream(device: torch.device) -> int:
    """The current stream; the tensors' GPU has to be the current one, where kernels are launched."""
    current = torch._C._cuda_getDevice()
    if current != device.index:
        raise ValueError(f"the tensors are on {device}, the current device is cuda:{current}")
    return torch._C._cuda_getCurrentRawStream(current)


def _positions(positions, rotary: Rotary, tokens: int, device: torch.device) -> int:
    """Checks int64 positions [tokens] (one axis) or [axes, tokens]; returns the axes' stride."""
    if not isinstance(rotary, Rotary):
        raise TypeError("rotary must be a Rotary")
    if not isinstance(positions, torch.Tensor):
        raise TypeError("positions must be a torch tensor")
    if positions.device != device or rotary.device != device:
        raise ValueError(f"positions are on {positions.device}, the rotary on {rotary.device}, expected {device}")
    if positions.dtype != torch.int64:
        raise TypeError(f"positions must be torch.int64, got {positions.dtype}")
    shape = positions.shape
    if shape != (rotary.axes, tokens) and (rotary.axes != 1 or shape != (tokens,)):
        raise ValueError(f"positions must be [{rotary.axes}, {tokens}], got {list(shape)}")
    if tokens > 1 and positions.stride(-1) != 1:
        raise ValueError("positions must be contiguous along the tokens")
    return positions.stride(0) if rotary.axes > 1 else 0


def _row_strides(t, name: str):
    """A strided [tokens, heads, head_dim] tensor whose rows the kernels read in 16-byte pieces; returns
    its dtype code and its token and head strides."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    dt = _dt(t)
    if t.dim() != 3:
        raise ValueError(f"{name} must be [tokens, heads, head_dim], got {list(t.shape)}")
    ts, hs, ds = t.stride()
    if t.shape[0] <= 1:  # the stride of a single token or head says nothing
        ts = 0
    if t.shape[1] <= 1:
        hs = 0
    if ds != 1 or (ts | hs) & (7 if dt == nvfp4.DTYPE_BF16 else 3) or t.data_ptr() & 15:
        raise ValueError(f"{name} must be contiguous along head_dim, every row at a multiple of 16 bytes")
    return dt, ts, hs


def _followed(t: torch.Tensor) -> bool:
    """Whether autograd follows t: backwards, or forwards by a tangent (in whatever mode)."""
    return t.requires_grad and torch.is_grad_enabled() or unpack_dual(t).tangent is not None


def _overwritten(t: torch.Tensor, name: str) -> None:
    """A tensor of the caller's is about to be written by a kernel. One that autograd follows would keep the
    history of what it held before, and is refused; what autograd saved of it counts as changed from here on."""
    if _followed(t):
        raise ValueError(f"{name} is followed by autograd and no gradient would flow to it: detach it, or call under "
                         "torch.no_grad()")
    if not t.is_inference():
        torch.autograd.graph.increment_version(t)


def _given_out(out, name: str, like):
    """Strides of an output that the caller gives, with like's shape and type."""
    if not isinstance(out, torch.Tensor) or out.shape != like.shape or out.dtype != like.dtype \
            or out.device != like.device:
        raise ValueError(f"{name} must be {like.dtype} {list(like.shape)} on {like.device}")
    _, ts, hs = _row_strides(out, name)
    _overwritten(out, name)
    return ts, hs


def _launch(x, positions, rotary: Rotary, transpose: bool, out=None):
    dt, ts, hs = _row_strides(x, "x")
    tokens, heads, hd = x.shape
    stride = _positions(positions, rotary, tokens, x.device)
    if hd % 8 or hd < 2 * rotary.pairs or hd > MAX_HEAD_DIM:
        raise ValueError(f"head_dim must be a multiple of 8 from {2 * rotary.pairs} to {MAX_HEAD_DIM}, got {hd}")
    if out is None:
        out = torch.empty((tokens, heads, hd), dtype=x.dtype, device=x.device)
        ots, ohs = heads * hd, hd
    else:
        ots, ohs = _given_out(out, "out", x)
    _check((_bound or lib()).nvfp4_rotate(
        rotary._ref, positions.data_ptr(), stride, x.data_ptr(), dt, tokens, heads, hd, ts, hs,
        out.data_ptr(), ots, ohs, int(transpose), _stream(x.device)), "nvfp4_rotate")
    return out


def _aligned(g):
    """The gradient itself where the kernel can read it, else a contiguous copy (an expanded one, say)."""
    ts, hs, ds = g.stride()
    if ds == 1 and not (g.data_ptr() | (ts | hs) * g.element_size()) & 15:
        return g
    return g.clone(memory_format=torch.contiguous_format)


class _Turned(torch.autograd.Function):
    """y = R x; dx = R^T dy, which is differentiable in turn. The tensors that make R are inputs so that they
    can be saved: a backward pass after one of them was changed is refused or, where saved-tensor hooks kept
    copies, takes those. Forward mode is not offered: torch refuses a tangent here."""

    @staticmethod
    def forward(ctx, x, positions, inv_freq, axis, rotary, transpose):
        ctx.save_for_backward(positions, inv_freq, axis)
        ctx.rotary, ctx.transpose = rotary, transpose
        return _launch(x, positions, rotary, transpose)

    @staticmethod
    def backward(ctx, gy):
        positions, inv_freq, axis = ctx.saved_tensors
        turn = _turned if _followed(gy) else _launch
        rotary = ctx.rotary._of(inv_freq, axis)
        return turn(_aligned(gy), positions, rotary, not ctx.transpose), None, None, None, None, None


def _turned(x, positions, rotary: Rotary, transpose: bool):
    return _Turned.apply(x, positions, rotary.inv_freq, rotary.axis, rotary, transpose)


def rotate(x: torch.Tensor, positions: torch.Tensor, rotary: Rotary, *, transpose: bool = False,
           out: torch.Tensor | None = None) -> torch.Tensor:
    """x [tokens, heads, head_dim] (bf16 or fp32, rows may be strided) turned by the tokens' positions
    (int64 [tokens], or [axes, tokens] with the rotary's axes). head_dim is a multiple of 8, at least
    2 * rotary.pairs. Queries and keys that lie beside each other in a fused projection can be turned
    in one call. With ``transpose`` the transposed matrix (for factor 1 the turn back). ``out`` may be x
    itself (in place) and must not be followed by autograd; without it gradients flow to x, backwards only: a
    tangent of forward mode is refused. As with any operator, a backward pass that is captured into a graph
    needs leaves that no eager graph still holds."""
    if isinstance(x, torch.Tensor) and _followed(x):
        if out is not None:
            raise ValueError("a call that needs gradients takes no out")
        return _turned(x, positions, rotary, transpose)
    return _launch(x, positions, rotary, transpose, out)
