"""Key/value cache in NVFP4: Python binding of the entry points of ``include/nvfp4_kv.h``.

A ``KVCache`` holds one layer's pages: packed E2M1 codes and E4M3 block scales of keys and
values, and one fp32 tensor scale per head. ``write`` quantises new keys and values into
cache slots, ``append`` does so with the keys turned by their positions on the way, ``read``
dequantises slots, ``attention`` attends over the cached tokens of each sequence and of a prefix
shared by the whole batch. As in ``nvfp4``, this module checks and
marshals arguments; the work is done by the HIP kernels on the current stream, there is
no CPU fallback, and no gradient flows through the results.

    cache = kvcache.KVCache.empty(pages, page_size, kv_heads, head_dim, S_k, S_v)
    kvcache.write(cache, k, v, slots)                       # slot = page * page_size + offset
    out = kvcache.attention(cache, q, block_table, kv_lens)  # one new token per sequence
"""
from __future__ import annotations

import ctypes
import operator

import torch

from . import nvfp4
from .nvfp4 import _I, _I64, _P, _SZ, _arg, _check, _dt, _Fixed, _need
from .rotary import Rotary, _given_out, _overwritten, _positions

MAX_HEAD_DIM = 1024            # write, read
MAX_ATTENTION_HEAD_DIM = 256
MAX_WINDOW = 1 << 30           # also sinks


class _Cache(ctypes.Structure):
    _fields_ = [("k_codes", _P), ("k_scales", _P), ("v_codes", _P), ("v_scales", _P),
                ("S_k", _P), ("S_v", _P),
                ("pages", _I64), ("page_size", _I64), ("kv_heads", _I64), ("head_dim", _I64)]


_SIGS = {
    "nvfp4_kv_write": (_I, [_P, _P, _P, _I, _I64, _I64, _I64, _I64, _I64, _P, _P]),
    "nvfp4_kv_append": (_I, [_P, _P, _P, _I64, _P, _P, _P, _I, _I64, _I64, _I64, _I64, _I64, _I64, _I64, _I64,
                             _P, _I64, _I64, _P, _P]),
    "nvfp4_kv_read": (_I, [_P, _P, _I64, _P, _P, _I, _P]),
    "nvfp4_kv_attention_workspace_size": (_SZ, [_P, _I, _I64, _I64, _I64, _I64, _I64, _I64]),
    "nvfp4_kv_attention": (_I, [_P, _P, _I, _I64, _I64, _I64, _I64, _I64, _P, _I64, _P, _I64, _P,
                                _I64, _P, _I64, ctypes.c_float, _I, _P, _P, _P, _SZ, _P]),
    "nvfp4_kv_window_attention_workspace_size": (_SZ, [_P, _I, _I64, _I64, _I64, _I64, _I64, _I64, _I64]),
    "nvfp4_kv_window_attention": (_I, [_P, _P, _I, _I64, _I64, _I64, _I64, _I64, _P, _I64, _P, _I64, _P, _I64,
                                       _I64, _I64, ctypes.c_float, _P, _P, _P, _SZ, _P]),
}
_bound = None


def lib():
    """libnvfp4 with the cache's entry points bound (raises if it was not built)."""
    global _bound
    if _bound is None:
        L = nvfp4.lib()
        for name, (res, args) in _SIGS.items():
            f = getattr(L, name)
            f.restype, f.argtypes = res, args
        _bound = L
    return _bound


class KVCache(_Fixed):
    """One layer's cache. Tensors (contiguous, on one GPU):
    k_codes, v_codes [pages, kv_heads, page_size, head_dim / 2] uint8;
    k_scales, v_scales [pages, kv_heads, page_size, head_dim / 16] uint8;
    S_k, S_v [kv_heads] fp32, the tensor scale of each head (amax / 2688 of calibration data).
    page_size is a power of two, 16 or more. Memory need not be initialised. The tensors may be changed between
    calls; an attribute cannot be replaced."""

    def __init__(self, k_codes, k_scales, v_codes, v_scales, S_k, S_v):
        _need(k_codes, "k_codes")
        if k_codes.dtype != torch.uint8 or k_codes.dim() != 4:
            raise ValueError("k_codes must be uint8 [pages, kv_heads, page_size, head_dim / 2]")
        pages, heads, size, half = k_codes.shape
        if size < 16 or size > 32768 or size & (size - 1):
            raise ValueError(f"page_size must be a power of two from 16 to 32768, got {size}")
        if half < 8 or half % 8 or 2 * half > MAX_HEAD_DIM:
            raise ValueError(f"head_dim must be a multiple of 16 up to {MAX_HEAD_DIM}, got {2 * half}")
        for t, name, last in ((k_scales, "k_scales", half // 8), (v_codes, "v_codes", half),
                              (v_scales, "v_scales", half // 8)):
            _arg(t, name, k_codes, torch.uint8)
            if tuple(t.shape) != (pages, heads, size, last):
                raise ValueError(f"{name} must be [{pages}, {heads}, {size}, {last}], got {list(t.shape)}")
        _arg(S_k, "S_k", k_codes, torch.float32, numel=heads)
        _arg(S_v, "S_v", k_codes, torch.float32, numel=heads)
        self.k_codes, self.k_scales, self.v_codes, self.v_scales = k_codes, k_scales, v_codes, v_scales
        self.S_k, self.S_v = S_k, S_v
        self.pages, self.kv_heads, self.page_size, self.head_dim = pages, heads, size, 2 * half
        self.device = k_codes.device
        self._index = self.device.index
        self._needs = {}  # attention's workspace size by the sizes of a call
        self._c = _Cache(*(t.data_ptr() for t in (k_codes, k_scales, v_codes, v_scales, S_k, S_v)),
                         pages, size, heads, 2 * half)
        self._ref = ctypes.addressof(self._c)

    @classmethod
    def empty(cls, pages: int, page_size: int, kv_heads: int, head_dim: int, S_k: torch.Tensor,
              S_v: torch.Tensor) -> "KVCache":
        """A cache of uninitialised pages on S_k's device."""
        def mem(last):
            return torch.empty(pages, kv_heads, page_size, last, dtype=torch.uint8, device=S_k.device)
        return cls(mem(head_dim // 2), mem(head_dim // 16), mem(head_dim // 2), mem(head_dim // 16),
                   S_k, S_v)


_BF16, _F32, _I32, _INT64 = torch.bfloat16, torch.float32, torch.int32, torch.int64


def _stream(cache: KVCache) -> int:
    """The current stream (without building a Stream object); the cache's GPU has to be
    the current one, where kernels are launched. torch's functions are looked up here, not at import:
    builds without GPU support lack them."""
    device = torch._C._cuda_getDevice()
    if device != cache._index:
        raise ValueError(f"the cache is on {cache.device}, the current device is cuda:{device}")
    return torch._C._cuda_getCurrentRawStream(cache._index)


def _rows(t, name: str, cache: KVCache, heads: int | None):
    """A strided [tokens, heads, head_dim] tensor whose rows the kernels read in 16-byte
    pieces; returns its dtype code and its token and head strides."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.device != cache.device:
        raise ValueError(f"{name} is on {t.device}, expected {cache.device}")
    dt = _dt(t)
    shape = t.shape
    if len(shape) != 3 or shape[2] != cache.head_dim or (heads is not None and shape[1] != heads):
        raise ValueError(f"{name} must be [tokens, {heads or 'heads'}, {cache.head_dim}], got {list(shape)}")
    ts, hs, ds = t.stride()
    if shape[0] <= 1:  # the stride of a single token or head says nothing
        ts = 0
    if shape[1] <= 1:
        hs = 0
    if ds != 1 or (ts | hs) & (7 if dt == nvfp4.DTYPE_BF16 else 3) or t.data_ptr() & 15:
        raise ValueError(f"{name} must be contiguous along head_dim, every row at a multiple of 16 bytes")
    return dt, ts, hs


def _ids(t, name: str, cache: KVCache, dim: int, dtype: torch.dtype = _I32):
    """A contiguous tensor of indices on the cache's GPU."""
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.dim() == dim and t.device == cache.device \
            and t.is_cuda and t.is_contiguous():
        return
    _need(t, name)
    if t.device != cache.device:
        raise ValueError(f"{name} is on {t.device}, expected {cache.device}")
    raise TypeError(f"{name} must be {dtype} with {dim} dimension{'s' if dim > 1 else ''}")


def write(cache: KVCache, k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor) -> None:
    """Quantise k, v [tokens, kv_heads, head_dim] (bf16 or fp32, rows may be strided) into the
    slots [tokens] (int64; page * page_size + offset; a slot outside the cache, e.g. -1, skips
    the token). Two tokens of one call must not share a slot."""
    dt, k_ts, k_hs = _rows(k, "k", cache, cache.kv_heads)
    v_dt, v_ts, v_hs = _rows(v, "v", cache, cache.kv_heads)
    if v_dt != dt:
        raise TypeError(f"v must be {k.dtype}, got {v.dtype}")
    n = k.shape[0]
    if v.shape[0] != n:
        raise ValueError(f"v must have {n} tokens, got {v.shape[0]}")
    _ids(slots, "slots", cache, 1, _INT64)
    if slots.shape[0] != n:
        raise ValueError(f"slots must have {n} elements, got {slots.shape[0]}")
    _check((_bound or lib()).nvfp4_kv_write(
        cache._ref, k.data_ptr(), v.data_ptr(), dt, n, k_ts, k_hs, v_ts, v_hs, slots.data_ptr(),
        _stream(cache)), "nvfp4_kv_write")


def append(cache: KVCache, k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor, positions: torch.Tensor,
           rotary: Rotary, q: torch.Tensor | None = None, *, q_out: torch.Tensor | None = None):
    """``write`` with k turned by the tokens' positions on the way (int64 [tokens], or [axes, tokens] with
    the rotary's axes; ``rotary.rotate`` without the rounding to k's type), v as it is. The rotary's
    pairs are a multiple of 8. Returns q [tokens, heads, head_dim] turned too, of every token, also
    of those that have no slot; None without q. ``q_out`` may be q itself (in place); one that autograd follows
    (q of a projection that is being trained) is refused outside of torch.no_grad(). One launch."""
    dt, k_ts, k_hs = _rows(k, "k", cache, cache.kv_heads)
    v_dt, v_ts, v_hs = _rows(v, "v", cache, cache.kv_heads)
    if v_dt != dt:
        raise TypeError(f"v must be {k.dtype}, got {v.dtype}")
    n = k.shape[0]
    if v.shape[0] != n:
        raise ValueError(f"v must have {n} tokens, got {v.shape[0]}")
    _ids(slots, "slots", cache, 1, _INT64)
    if slots.shape[0] != n:
        raise ValueError(f"slots must have {n} elements, got {slots.shape[0]}")
    p_stride = _positions(positions, rotary, n, cache.device)
    if rotary.pairs % 8 or 2 * rotary.pairs > cache.head_dim:
        raise ValueError(f"the rotary's pairs must be a multiple of 8 up to {cache.head_dim // 2}, got {rotary.pairs}")
    heads = q_ts = q_hs = o_ts = o_hs = 0
    if q is not None:
        q_dt, q_ts, q_hs = _rows(q, "q", cache, None)
        if q_dt != dt:
            raise TypeError(f"q must be {k.dtype}, got {q.dtype}")
        if q.shape[0] != n:
            raise ValueError(f"q must have {n} tokens, got {q.shape[0]}")
        heads = q.shape[1]
        if q_out is None:
            q_out = torch.empty((n, heads, cache.head_dim), dtype=q.dtype, device=q.device)
            o_ts, o_hs = heads * cache.head_dim, cache.head_dim
        else:
            o_ts, o_hs = _given_out(q_out, "q_out", q)
    elif q_out is not None:
        raise ValueError("q_out without q")
    _check((_bound or lib()).nvfp4_kv_append(
        cache._ref, rotary._ref, positions.data_ptr(), p_stride, None if q is None else q.data_ptr(),
        k.data_ptr(), v.data_ptr(), dt, n, heads, q_ts, q_hs, k_ts, k_hs, v_ts, v_hs,
        None if q is None else q_out.data_ptr(), o_ts, o_hs, slots.data_ptr(), _stream(cache)), "nvfp4_kv_append")
    return q_out


def read(cache: KVCache, slots: torch.Tensor, dtype: torch.dtype = torch.bfloat16):
    """Keys and values [n, kv_heads, head_dim] of the slots [n] (int64), dequantised to `dtype`;
    zeros for slots outside the cache."""
    _ids(slots, "slots", cache, 1, _INT64)
    if dtype is not _BF16 and dtype is not _F32:
        raise TypeError(f"unsupported dtype {dtype} (bf16 or fp32)")
    n = slots.shape[0]
    k = torch.empty((n, cache.kv_heads, cache.head_dim), dtype=dtype, device=cache.device)
    v = torch.empty_like(k)
    _check((_bound or lib()).nvfp4_kv_read(
        cache._ref, slots.data_ptr(), n, k.data_ptr(), v.data_ptr(), _dt(k), _stream(cache)), "nvfp4_kv_read")
    return k, v


def attention_workspace_size(cache: KVCache, dtype: torch.dtype, tokens: int, heads: int, batch: int,
                             max_q: int, max_kv: int, prefix_len: int = 0, *, window: int | None = None,
                             sinks: int = 0) -> int:
    """Bytes of workspace that `attention` needs for these sizes."""
    dt = nvfp4.DTYPE_BF16 if dtype == torch.bfloat16 else nvfp4.DTYPE_F32
    if window is not None:
        return int(lib().nvfp4_kv_window_attention_workspace_size(cache._ref, dt, tokens, heads, batch, max_q,
                                                                  max_kv, window, sinks))
    return int(lib().nvfp4_kv_attention_workspace_size(cache._ref, dt, tokens, heads, batch, max_q,
                                                       max_kv, prefix_len))


def attention(cache: KVCache, q: torch.Tensor, block_table: torch.Tensor | None = None,
              kv_lens: torch.Tensor | None = None, *, q_offsets: torch.Tensor | None = None,
              max_q: int | None = None, max_kv: int | None = None,
              prefix_pages: torch.Tensor | None = None, prefix_len: int = 0,
              scale: float | None = None, causal: bool = True, window: int | None = None, sinks: int = 0,
              out: torch.Tensor | None = None, return_lse: bool = False,
              workspace: torch.Tensor | None = None):
    """Softmax attention of q [tokens, heads, head_dim] (bf16 or fp32, rows may be strided) over
    cached tokens; query head j reads key/value head j // (heads // kv_heads).

    The tokens are the batch's sequences packed: q_offsets [batch + 1] (int32), at most max_q
    each; without q_offsets every sequence has tokens / batch. A query sees the first
    prefix_len tokens of prefix_pages (int32, one list for the whole batch), and of its own
    sequence the kv_lens[b] (int32 [batch], at most max_kv) tokens in the pages
    block_table[b] (int32 [batch, width]): with n query tokens, token i sees its own tokens
    j <= kv_lens[b] - n + i if `causal`, all of them otherwise. max_q defaults to tokens and
    max_kv to width * page_size; smaller true bounds save work. scale defaults to
    head_dim ** -0.5.

    With `window`, a query at position P = kv_lens[b] - n + i sees the tokens t <= P with t > P - window,
    and the first `sinks` tokens up to its own. Only those are read: pages between them may be gone
    from the block table. A window is causal and takes no prefix (a prompt that all share can stand in
    every block table).

    Returns out [tokens, heads, head_dim] in q's dtype (zeros for a query that sees nothing),
    and with return_lse also lse [tokens, heads] fp32 (the logarithm of the softmax sum; -inf for
    such a query). `out` (contiguous, of q's type and size) must not be followed by autograd. `workspace`
    (uint8, attention_workspace_size bytes) saves an allocation."""
    dt, q_ts, q_hs = _rows(q, "q", cache, None)
    tokens, heads, hd = q.shape
    if hd > MAX_ATTENTION_HEAD_DIM:
        raise ValueError(f"attention takes head_dim up to {MAX_ATTENTION_HEAD_DIM}, got {hd}")
    if heads and (not cache.kv_heads or heads % cache.kv_heads):
        raise ValueError(f"{heads} query heads are no multiple of {cache.kv_heads} key/value heads")
    batch, width = 1, 0
    if (block_table is None) != (kv_lens is None):
        raise ValueError("block_table and kv_lens belong together")
    if block_table is not None:
        _ids(block_table, "block_table", cache, 2)
        batch, width = block_table.shape
        _ids(kv_lens, "kv_lens", cache, 1)
        if kv_lens.shape[0] != batch:
            raise ValueError(f"kv_lens must have {batch} elements, got {kv_lens.shape[0]}")
    if q_offsets is not None:
        _ids(q_offsets, "q_offsets", cache, 1)
        n = q_offsets.shape[0] - 1
        if n < 0 or (block_table is not None and n != batch):
            raise ValueError(f"q_offsets must have {batch + 1} elements, got {n + 1}")
        batch = n
        max_q = tokens if max_q is None else min(int(max_q), tokens)
    else:
        if (tokens % batch if batch else tokens):
            raise ValueError(f"{tokens} tokens are no multiple of {batch} sequences: give q_offsets")
        if max_q is not None and batch and max_q != tokens // batch:
            raise ValueError(f"without q_offsets max_q is tokens / batch = {tokens // batch}, got {max_q}")
        max_q = tokens // batch if batch else 0
    room = width * cache.page_size
    max_kv = room if max_kv is None else min(int(max_kv), room)
    if max_q < 0 or max_kv < 0 or prefix_len < 0:
        raise ValueError("max_q, max_kv and prefix_len must not be negative")
    if window is not None:
        if not causal or prefix_len:
            raise ValueError("a window is causal and takes no prefix")
        window, sinks = operator.index(window), operator.index(sinks)
        if not 1 <= window <= MAX_WINDOW or not 0 <= sinks <= MAX_WINDOW:
            raise ValueError(f"window must be 1 to 2^30 and sinks 0 to 2^30, got {window} and {sinks}")
    elif sinks:
        raise ValueError("sinks without a window")
    pages = None
    if prefix_len:
        _ids(prefix_pages, "prefix_pages", cache, 1)
        if prefix_pages.shape[0] * cache.page_size < prefix_len:
            raise ValueError(f"{prefix_pages.shape[0]} prefix pages hold fewer than {prefix_len} tokens")
        pages = prefix_pages.data_ptr()
    if out is None:
        out = torch.empty(tokens, heads, hd, dtype=q.dtype, device=q.device)
    else:
        _arg(out, "out", q, q.dtype, numel=q.numel())
        _overwritten(out, "out")
    lse = torch.empty(tokens, heads, dtype=torch.float32, device=q.device) if return_lse else None
    L = _bound or lib()
    if window is None:
        sizes, size_of = (dt, tokens, heads, batch, max_q, max_kv, prefix_len), L.nvfp4_kv_attention_workspace_size
    else:
        sizes = (dt, tokens, heads, batch, max_q, max_kv, window, sinks)
        size_of = L.nvfp4_kv_window_attention_workspace_size
    need = cache._needs.get(sizes)
    if need is None:
        if len(cache._needs) >= 4096:
            cache._needs.clear()
        need = cache._needs[sizes] = size_of(cache._ref, *sizes)
    if workspace is not None:
        _arg(workspace, "workspace", cache.k_codes, torch.uint8, min_numel=need)
    elif need:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    scale = hd ** -0.5 if scale is None else scale
    offsets = None if q_offsets is None else q_offsets.data_ptr()
    table = None if block_table is None else block_table.data_ptr()
    lens = None if kv_lens is None else kv_lens.data_ptr()
    ends = (out.data_ptr(), None if lse is None else lse.data_ptr(),
            None if workspace is None else workspace.data_ptr(),
            0 if workspace is None else workspace.numel(), _stream(cache))
    if window is None:
        _check(L.nvfp4_kv_attention(
            cache._ref, q.data_ptr(), dt, tokens, heads, q_ts, q_hs, batch, offsets, max_q, table, width, lens,
            max_kv, pages, prefix_len, scale, int(causal), *ends), "nvfp4_kv_attention")
    else:
        _check(L.nvfp4_kv_window_attention(
            cache._ref, q.data_ptr(), dt, tokens, heads, q_ts, q_hs, batch, offsets, max_q, table, width, lens,
            max_kv, window, sinks, scale, *ends), "nvfp4_kv_window_attention")
    return (out, lse) if return_lse else out
