"""Paged key/value cache: answering with a model that this library trained.

    cache = PagedCache(num_pages, 64, Hkv, 128, num_layers=32, max_seqs=256)
    cache.resize([0], [prompt_len])                          # pages for sequence 0
    table, kv_len = cache.tables([0], device="cuda")         # int32 [1, W], [1]
    for layer in range(32):
        q = cache.append(k, v, table, cu_q, kv_len, layer=layer, rope=rope, pos=pos, q=q)   # rotate, write
        o = cache.attend(q, table, cu_q, kv_len, max_q, layer=layer)
    cache.fork(0, 1)                                         # sequence 1 shares sequence 0's pages

A step of single tokens is the same three calls with one row per sequence. Everything that changes from step to step is
read on the device, so append and attend can be captured in a CUDA graph (after one eager call each) and replayed.
include/anchorattn.h states each call's layouts and rules ("Paged key/value cache"); the mask is AnchorAttention's ("When
Precision Meets Position", architecture page, §3.4 "AnchorAttention: The Shared Anchor Design"). Like the rest of
the binding this marshals arguments: every step runs in the library.
"""
from __future__ import annotations

import ctypes
import struct

import numpy as np
import torch

from .axes import _check_rows, _check_tensor, _on, _out, _rows
from .binding import AACacheConfig, _check, _stream_ptr, lib

__all__ = ["PagedCache"]


_BATCH = struct.Struct("@3P4i")  # aa_cache_batch


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
    """The pool of pages, bf16 [num_layers, num_pages, Hkv, page_size, D] for keys and for values, and which sequence holds
    which page. k_pages / v_pages: tensors to use as the pool (else allocated, uncleared, on `device`). max_seqs = 0: no
    bookkeeping, the caller has page tables of its own."""

    def __init__(self, num_pages, page_size, num_kv_heads, head_dim, num_layers=1, max_seqs=0, k_pages=None, v_pages=None,
                 device=None, host_only=False):
        self.cfg = AACacheConfig(int(num_layers), int(num_pages), int(page_size), int(num_kv_heads), int(head_dim),
                                 int(max_seqs), int(bool(host_only)))
        self.L, self.P, self.ps = int(num_layers), int(num_pages), int(page_size)
        self.Hkv, self.D, self.host_only = int(num_kv_heads), int(head_dim), bool(host_only)
        self._h = None
        h = ctypes.c_void_p()
        if host_only:
            _check(lib().aa_cache_create(ctypes.addressof(self.cfg), None, None, ctypes.byref(h)))
            self.k_pages = self.v_pages = self.device = None
            self._h = h
            return
        shape = (self.L, self.P, self.Hkv, self.ps, self.D)
        if (k_pages is None) != (v_pages is None):
            raise ValueError("give both k_pages and v_pages or neither")
        if k_pages is None:
            if min(shape) < 1:
                raise ValueError("sizes must be >= 1")
            dev = torch.device("cuda" if device is None else device)
            k_pages = torch.empty(shape, dtype=torch.bfloat16, device=dev)
            v_pages = torch.empty(shape, dtype=torch.bfloat16, device=dev)
        elif device is not None:
            raise ValueError("device goes without k_pages and v_pages")
        for name, x in (("k_pages", k_pages), ("v_pages", v_pages)):
            if not isinstance(x, torch.Tensor) or not x.is_cuda:
                raise ValueError(f"{name} must be a CUDA tensor")
            _check_tensor(name, x, shape, torch.bfloat16, k_pages.device)
        self.k_pages, self.v_pages, self.device = k_pages, v_pages, k_pages.device
        with torch.cuda.device(self.device):
            _check(lib().aa_cache_create(ctypes.addressof(self.cfg), k_pages.data_ptr(), v_pages.data_ptr(),
                                         ctypes.byref(h)))
        self._h = h

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

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    def _stream(self, stream):
        return None if self.host_only else _stream_ptr(stream, self.device.index)

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
        if a.size != b.size:
            raise ValueError("src and dst must have the same number of entries")
        _check(lib().aa_cache_copy_pages(self._h, a.ctypes.data, b.ctypes.data, a.size, self._stream(stream)))

    def check_device_error(self, stream=None):
        _check(lib().aa_cache_check_error(self._h, self._stream(stream)))

    def _batch(self, page_table, cu_q, kv_len, T, layer):
        """aa_cache_batch as bytes."""
        dev = self.device
        if dev is None:
            raise ValueError("the cache was created with host_only = True")
        for x, name in ((page_table, "page_table"), (cu_q, "cu_q"), (kv_len, "kv_len")):
            if not isinstance(x, torch.Tensor) or x.dtype is not torch.int32 or x.device != dev or not x.is_contiguous():
                raise ValueError(f"{name} must be a contiguous int32 tensor on {dev}")
        shape = page_table.shape
        if len(shape) != 2 or cu_q.shape != (shape[0] + 1,) or kv_len.shape != (shape[0],):
            raise ValueError(f"page_table [B, W], cu_q [B + 1] and kv_len [B] do not fit together: {tuple(shape)}, "
                             f"{tuple(cu_q.shape)}, {tuple(kv_len.shape)}")
        return _BATCH.pack(page_table.data_ptr(), cu_q.data_ptr(), kv_len.data_ptr(), shape[0], shape[1], T, layer)

    def append(self, k, v, page_table, cu_q, kv_len, layer=0, rope=None, pos=None, q=None, out_q=None, stream=None):
        """Write the new tokens' k (rotated by rope at pos) and v [T, Hkv, D] to their pages; with q [T, Hq, D] the same
        launch rotates q, and the result is returned."""
        dev, D = self.device, self.D
        _check_rows("k", k, None, self.Hkv, D, dev)
        T = k.shape[0]
        _check_rows("v", v, T, self.Hkv, D, dev)
        batch = self._batch(page_table, cu_q, kv_len, T, layer)
        if (rope is None) != (pos is None):
            raise ValueError("give both rope and pos or neither")
        if q is None:
            if out_q is not None:
                raise ValueError("out_q goes with q")
        else:
            _check_rows("q", q, T, None, D, dev)
            if rope is None:
                raise ValueError("q is rotated: it needs rope and pos")
        with _on(stream):
            k, sk = _rows(k)
            v, sv = _rows(v)
            rp, pp = None, None
            if rope is not None:
                pos = rope._positions(pos, T, dev)
                rp, pp = rope._at, pos.data_ptr()
            yq, qp, yp, sq, hq = None, None, None, 0, 0
            if q is not None:
                yq = _out("out_q", out_q, q)
                q, sq = _rows(q)
                qp, yp, hq = q.data_ptr(), yq.data_ptr(), q.shape[1]
            status = lib().aa_cache_append(self._h, batch, k.data_ptr(), sk, v.data_ptr(), sv, rp, pp, qp, sq, yp, hq,
                                           _stream_ptr(stream, dev.index))
            if status:
                _check(status)
        return yq

    def workspace_bytes(self, num_seqs, total_tokens, max_q, table_width, q_heads):
        return int(lib().aa_cache_attend_workspace_bytes(self._h, int(num_seqs), int(total_tokens), int(max_q),
                                                         int(table_width), int(q_heads)))

    def alloc_workspace(self, num_seqs, total_tokens, max_q, table_width, q_heads):
        """Scratch for attend calls of these sizes, one for each that may overlap with another."""
        n = self.workspace_bytes(num_seqs, total_tokens, max_q, table_width, q_heads)
        return torch.empty(max(n, 256), device=self.device, dtype=torch.uint8)

    def attend(self, q, page_table, cu_q, kv_len, max_q, layer=0, key_lo=None, anchor=False, softmax_scale=0.0, out=None,
               lse=None, workspace=None, return_lse=False, stream=None):
        """Attention of the new tokens' rotated q [T, Hq, D] over their sequences' pages: o [T, Hq, D], and with
        return_lse the log-sum-exp [Hq, T] fp32. key_lo: int32 [T], the first key each row sees; anchor: key 0 is seen too."""
        dev = self.device
        _check_rows("q", q, None, None, self.D, dev)
        T, hq, _ = q.shape
        batch = self._batch(page_table, cu_q, kv_len, T, layer)
        with _on(stream):
            kp = None
            if key_lo is not None:
                if not isinstance(key_lo, torch.Tensor) or key_lo.dtype is not torch.int32 or key_lo.device != dev \
                        or key_lo.shape != (T,):
                    raise ValueError(f"key_lo must be an int32 tensor [{T}] on {dev}")
                key_lo = key_lo.contiguous()
                kp = key_lo.data_ptr()
            o = _out("out", out, q)
            if lse is not None:
                _check_tensor("lse", lse, (hq, T), torch.float32, dev)
            elif return_lse:
                lse = torch.empty((hq, T), dtype=torch.float32, device=dev)
            if workspace is None:
                workspace = self.alloc_workspace(page_table.shape[0], T, max_q, page_table.shape[1], hq)
            elif not isinstance(workspace, torch.Tensor) or workspace.dtype is not torch.uint8 or workspace.device != dev \
                    or not workspace.is_contiguous():
                raise ValueError(f"workspace must be a contiguous uint8 tensor on {dev}")
            q, sq = _rows(q)
            status = lib().aa_cache_attend(self._h, batch, q.data_ptr(), sq, hq, max_q, kp, 1 if anchor else 0,
                                           softmax_scale or 0.0, o.data_ptr(), None if lse is None else lse.data_ptr(),
                                           workspace.data_ptr(), workspace.numel(), _stream_ptr(stream, dev.index))
            if status:
                _check(status)
        return (o, lse) if return_lse else o
