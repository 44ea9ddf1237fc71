"""Paged key/value cache: answering with a model that this library trained.

    cache = PagedCache(num_pages, 64, Hkv, 128, num_layers=32, max_seqs=256)
    cache.resize([0], [prompt_len])                          # pages for sequence 0
    table, kv_len = cache.tables([0], device="cuda")         # int32 [1, W], [1]
    for layer in range(32):
        q = cache.append(k, v, table, cu_q, kv_len, layer=layer, rope=rope, pos=pos, q=q)   # rotate, write
        o = cache.attend(q, table, cu_q, kv_len, max_q, layer=layer)
    cache.fork(0, 1)                                         # sequence 1 shares sequence 0's pages

PagedCache(..., dtype=torch.float8_e4m3fn) keeps the pages in 8 bits, quantised as append writes them: half of the memory
and of what a decoding step reads. All calls are the same; read gives back what the pages hold.

A step of drafted trees, verified in one pass:

    mask, pos = cache.tree_masks(parents, cu_q, kv_len, max_q)    # from each drafted token's parent
    for layer in range(32):
        q = cache.append(k, v, table, cu_q, kv_len, layer=layer, rope=rope, pos=pos, q=q)
        o = cache.attend(q, table, cu_q, kv_len, max_q, layer=layer, tree=mask)
    cache.accept(table, cu_q, kv_len, path)                       # the kept tokens' indices, -1 behind them
    cache.resize([0], [base + kept])

A step of single tokens is the same three calls with one row per sequence. Everything that changes from step to step is
read on the device, so append and attend can be captured in a CUDA graph (after one eager call each) and replayed.
append and attend are for answering: their results carry no gradient (rope_axes and anchor_attention's do).
A call on a stream other than the current one reads its inputs there: the caller keeps them until it has run
(Tensor.record_stream).
resize and free work on the host, in time that grows with the pool: a step of 64 sequences 11 us with 4K pages, 27
with 64K; giving a sequence back 19 and 226 us.
include/anchorattn.h states each call's layouts and rules ("Paged key/value cache"); the mask is AnchorAttention's ("When
Precision Meets Position", architecture page, §3.4 "AnchorAttention: The Shared Anchor Design"). Like the rest of
the binding this marshals arguments: every step runs in the library.
"""
from __future__ import annotations

import ctypes

import numpy as np
import torch

from .binding import AACacheConfig, _check, _stream, lib, native

__all__ = ["PagedCache"]


def _host_i32(name, x):
    if type(x) is np.ndarray and x.dtype == np.int32 and x.ndim == 1 and x.flags.c_contiguous:
        return x
    a = np.ascontiguousarray(np.asarray(x))
    if a.ndim != 1 or (a.size and a.dtype.kind not in "iu"):
        raise ValueError(f"{name} must be a list of integers")
    if a.size and (a.min() < -2 ** 31 or a.max() >= 2 ** 31):
        raise ValueError(f"{name} must hold 32-bit integers")
    return np.ascontiguousarray(a, dtype=np.int32)


def _i32p(a):
    return a.ctypes.data_as(ctypes.POINTER(ctypes.c_int32))


class PagedCache:
    """The pool of pages, [num_layers, num_pages, Hkv, page_size, D] for keys and for values, and which sequence holds
    which page. dtype: torch.bfloat16, or torch.float8_e4m3fn for 8-bit pages with k_scales / v_scales, float8_e8m0fnu
    [num_layers, num_pages, Hkv, page_size] (a token's power of two, 2^-124 to 2^119 or NaN: page value * scale is what it
    stands for). k_pages / v_pages (and the scales): tensors to use as the pool, whose type they give (else allocated,
    uncleared, on `device`). max_seqs = 0: no bookkeeping, the caller has page tables of its own."""

    def __init__(self, num_pages, page_size, num_kv_heads, head_dim, num_layers=1, max_seqs=0, k_pages=None, v_pages=None,
                 device=None, host_only=False, dtype=None, k_scales=None, v_scales=None):
        self._h, self._dev = None, -1
        self.cfg = AACacheConfig(int(num_layers), int(num_pages), int(page_size), int(num_kv_heads), int(head_dim),
                                 int(max_seqs), int(bool(host_only)))
        self.L, self.P, self.ps = int(num_layers), int(num_pages), int(page_size)
        self.Hkv, self.D, self.host_only = int(num_kv_heads), int(head_dim), bool(host_only)
        h = ctypes.c_void_p()
        if dtype is None:
            dtype = k_pages.dtype if isinstance(k_pages, torch.Tensor) else torch.bfloat16
        if dtype not in (torch.bfloat16, torch.float8_e4m3fn):
            raise ValueError(f"dtype must be torch.bfloat16 or torch.float8_e4m3fn, got {dtype}")
        self.dtype, fp8 = dtype, dtype == torch.float8_e4m3fn
        if host_only:
            _check(lib().aa_cache_create(ctypes.addressof(self.cfg), None, None, ctypes.byref(h)))
            self.k_pages = self.v_pages = self.k_scales = self.v_scales = self.device = None
            self._h, self._dev = h, -1
            return
        shape = (self.L, self.P, self.Hkv, self.ps, self.D)
        if (k_pages is None) != (v_pages is None):
            raise ValueError("give both k_pages and v_pages or neither")
        if any((x is not None) != (fp8 and k_pages is not None) for x in (k_scales, v_scales)):
            raise ValueError("k_scales and v_scales go with 8-bit k_pages and v_pages")
        if k_pages is None:
            if min(shape) < 1:
                raise ValueError("sizes must be >= 1")
            dev = torch.device("cuda" if device is None else device)
            k_pages = torch.empty(shape, dtype=dtype, device=dev)
            v_pages = torch.empty(shape, dtype=dtype, device=dev)
            if fp8:
                k_scales, v_scales = (torch.empty(shape[:-1], dtype=torch.uint8, device=dev).view(torch.float8_e8m0fnu)
                                      for _ in range(2))
        elif device is not None:
            raise ValueError("device goes without k_pages and v_pages")
        pool = [("k_pages", k_pages, dtype, shape), ("v_pages", v_pages, dtype, shape)]
        if fp8:
            pool += [("k_scales", k_scales, torch.float8_e8m0fnu, shape[:-1]),
                     ("v_scales", v_scales, torch.float8_e8m0fnu, shape[:-1])]
        for name, x, kind, size in pool:
            if not isinstance(x, torch.Tensor) or not x.is_cuda or x.dtype != kind or x.device != k_pages.device:
                raise ValueError(f"{name} must be a {str(kind)[6:]} CUDA tensor, all on one device")
            if x.shape != size or not x.is_contiguous():
                raise ValueError(f"{name} must be contiguous with shape {size}, got {tuple(x.shape)}")
        self.k_pages, self.v_pages, self.device = k_pages, v_pages, k_pages.device
        self.k_scales, self.v_scales = k_scales, v_scales
        with torch.cuda.device(self.device):
            if fp8:
                _check(lib().aa_cache_create_fp8(ctypes.addressof(self.cfg), k_pages.data_ptr(), k_scales.data_ptr(),
                                                 v_pages.data_ptr(), v_scales.data_ptr(), ctypes.byref(h)))
            else:
                _check(lib().aa_cache_create(ctypes.addressof(self.cfg), k_pages.data_ptr(), v_pages.data_ptr(),
                                             ctypes.byref(h)))
        self._h, self._dev = h, self.device.index

    # ---- lifetime
    def close(self):
        if getattr(self, "_h", None):
            lib().aa_cache_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def __reduce__(self):  # copy.copy and copy.deepcopy ask it too
        raise TypeError("a PagedCache owns its handle: it cannot be copied or pickled")

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    def _stream(self, stream):
        return None if self.host_only else _stream(stream)

    # ---- bookkeeping (host)
    def resize(self, seqs, lens, stream=None):
        """Set the lengths of the sequences (growing takes pages, shrinking gives them back); all or nothing."""
        s, n = _host_i32("seqs", seqs), _host_i32("lens", lens)
        if s.size != n.size:
            raise ValueError("seqs and lens must have the same number of entries")
        _check(lib().aa_cache_resize(self._h, _i32p(s), _i32p(n), s.size, self._stream(stream)))

    def free(self, seqs, stream=None):
        """Give the sequences' pages back: resize to 0."""
        s = _host_i32("seqs", seqs)
        self.resize(s, np.zeros_like(s), stream)

    def fork(self, src, dst):
        """Sequence dst (empty) shares src's pages from here on."""
        _check(lib().aa_cache_fork(self._h, int(src), int(dst)))

    def compact(self, stream=None):
        """Move the pages in use to the front of the pool; returns how many moved. Tables taken before are stale."""
        n = ctypes.c_int32()
        _check(lib().aa_cache_compact(self._h, self._stream(stream), ctypes.byref(n)))
        return n.value

    def stats(self):
        a, b, c = ctypes.c_int32(), ctypes.c_int32(), ctypes.c_int32()
        _check(lib().aa_cache_stats(self._h, ctypes.byref(a), ctypes.byref(b), ctypes.byref(c)))
        return {"free_pages": a.value, "shared_pages": b.value, "longest": c.value}

    def tables(self, seqs, width=None, device=None):
        """Page tables int32 [n, width] (entries past the last page -1) and lengths int32 [n] of the sequences: numpy arrays,
        or tensors on `device`. width defaults to the longest of them."""
        s = _host_i32("seqs", seqs)
        lens = np.zeros(s.size, dtype=np.int32)
        _check(lib().aa_cache_tables(self._h, _i32p(s), s.size, None, 0, _i32p(lens)))
        if width is None:
            width = max(1, -(-int(lens.max(initial=0)) // self.ps))
        table = np.empty((s.size, int(width)), dtype=np.int32)
        _check(lib().aa_cache_tables(self._h, _i32p(s), s.size, _i32p(table), int(width), _i32p(lens)))
        if device is None:
            return table, lens
        return torch.from_numpy(table).to(device), torch.from_numpy(lens).to(device)

    # ---- device calls
    def copy_pages(self, src, dst, stream=None):
        """Copy page src[i] to dst[i] (host integers), all layers, keys and values."""
        a, b = _host_i32("src", src), _host_i32("dst", dst)
        r = native().cache_copy_pages(self._h.value if self._h else 0, self._dev, a, b, stream)
        if r:
            _check(r)

    def check_device_error(self, stream=None):
        _check(lib().aa_cache_check_error(self._h, self._stream(stream)))

    def _device_handle(self):
        """The handle's address, for the native calls."""
        if self._dev < 0 or self._h is None:
            raise ValueError("the cache is closed or was created with host_only = True")
        return self._h.value

    def append(self, k, v, page_table, cu_q, kv_len, layer=0, rope=None, pos=None, q=None, out_q=None, stream=None):
        """Write the new tokens' k (rotated by rope at pos) and v [T, Hkv, D] to their pages; with q [T, Hq, D] the same
        launch rotates q, and the result is returned."""
        r = native().cache_append(self._device_handle(), self._dev, self.Hkv, self.D, k, v, page_table, cu_q, kv_len, layer,
                                  None if rope is None else rope._at, 0 if rope is None else rope.num_axes, pos, q, out_q,
                                  stream)
        if type(r) is int:
            _check(r)
        return r

    def read(self, page_table, cu_q, kv_len, total_tokens, layer=0, out_k=None, out_v=None, stream=None):
        """What the pages hold of the new tokens: k (as stored, rotated) and v, bf16 [total_tokens, Hkv, D]. Rows outside
        the batch are not written."""
        r = native().cache_read(self._device_handle(), self._dev, self.Hkv, self.D, page_table, cu_q, kv_len, total_tokens,
                                layer, out_k, out_v, stream)
        if type(r) is int:
            _check(r)
        return r

    def tree_masks(self, parents, cu_q, kv_len, max_q, out_mask=None, out_pos=None, stream=None):
        """Masks int64 [T, ceil(max_q / 64)] and positions int32 [T] of drafted trees, for attend's tree and append's pos.
        parents: int32 [T], each new token's parent among its sequence's new tokens before it, -1: the cached tokens.
        Unlike attend's, this max_q is no hint: tokens of a sequence at and behind the masks' width are in no mask, their
        own included."""
        r = native().cache_tree_masks(self._device_handle(), self._dev, parents, cu_q, kv_len, max_q, out_mask, out_pos, stream)
        if type(r) is int:
            _check(r)
        return r

    def accept(self, page_table, cu_q, kv_len, path, stream=None):
        """Move the kept new tokens' keys and values up behind the cached tokens, in all layers: token path[b, i] to place i.
        path: int32 [B, any], ascending indices among the sequence's new tokens, negative behind the last."""
        r = native().cache_accept(self._device_handle(), self._dev, page_table, cu_q, kv_len, path, stream)
        if r:
            _check(r)

    def workspace_bytes(self, num_seqs, total_tokens, max_q, table_width, q_heads):
        return int(lib().aa_cache_attend_workspace_bytes(self._h, int(num_seqs), int(total_tokens), int(max_q),
                                                         int(table_width), int(q_heads)))

    def alloc_workspace(self, num_seqs, total_tokens, max_q, table_width, q_heads):
        """Scratch for attend calls of these sizes, one for each that may overlap with another."""
        n = self.workspace_bytes(num_seqs, total_tokens, max_q, table_width, q_heads)
        return torch.empty(max(n, 256), device=self.device, dtype=torch.uint8)

    def attend(self, q, page_table, cu_q, kv_len, max_q, layer=0, key_lo=None, anchor=False, softmax_scale=0.0, out=None,
               lse=None, workspace=None, return_lse=False, stream=None, tree=None):
        """Attention of the new tokens' rotated q [T, Hq, D] over their sequences' pages: o [T, Hq, D], and with
        return_lse the log-sum-exp [Hq, T] fp32. key_lo: int32 [T], the first key each row sees; anchor: key 0 is seen too.
        tree: int64 [T, words], drafted trees: bit c % 64 of word c // 64 says whether the row sees new token c of its
        sequence (tree_masks makes them of parents); of the cached ones it sees all from key_lo on."""
        r = native().cache_attend(self._device_handle(), self._dev, self.D, q, page_table, cu_q, kv_len, max_q, layer, key_lo,
                                  anchor, softmax_scale or 0.0, out, lse, workspace, return_lse, tree, stream)
        if type(r) is int:
            _check(r)
        return r
