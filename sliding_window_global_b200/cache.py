"""ctypes binding of the paged cache (swa_cache_append / swa_cache_attend).

Argument marshalling only, as in ``swa.py``: rotation, norm and attention run in the
library's CUDA kernels, and a call on anything but CUDA tensors raises.
"""
from __future__ import annotations

import ctypes
from typing import Optional

import torch

from .rotary import (F, I, I64, NO_ROTATION, P, HeadNorm, Rotary, Rotation, check_fp32, check_index, check_rows,
                     current_stream, elsewhere, head_norm, packer)
from .swa import SwaError, _dtype_code, load_library


class Cache(ctypes.Structure):
    """swa_cache of include/swa.h."""
    _fields_ = [("k_pages", P), ("v_pages", P), ("num_pages", I), ("num_kv_heads", I), ("page_size", I),
                ("head_dim", I), ("dtype", I), ("error_word", P)]


class CacheBatch(ctypes.Structure):
    """swa_cache_batch of include/swa.h."""
    _fields_ = [("batch", I), ("num_tokens", I), ("block_table", P), ("max_pages", I), ("seq_lens", P),
                ("cu_tokens", P)]


class CacheAppendArgs(ctypes.Structure):
    """swa_cache_append_args of include/swa.h (each stride array as its elements)."""
    _fields_ = [
        ("num_q_heads", I), ("q", P), ("k", P), ("v", P), ("q_stride0", I64), ("q_stride1", I64),
        ("k_stride0", I64), ("k_stride1", I64), ("v_stride0", I64), ("v_stride1", I64), ("q_out", P),
        ("q_out_stride0", I64), ("q_out_stride1", I64), ("rotation", Rotation), ("head_norm", HeadNorm),
    ]


class CacheAttendArgs(ctypes.Structure):
    """swa_cache_attend_args of include/swa.h (the stride array as its elements)."""
    _fields_ = [
        ("num_q_heads", I), ("q", P), ("q_stride0", I64), ("q_stride1", I64), ("max_tokens", I), ("max_len", I),
        ("window", I), ("softcap", F), ("scale", F), ("out", P), ("lse", P), ("workspace", P),
        ("workspace_bytes", ctypes.c_size_t),
    ]


_pack_batch, _pack_append, _pack_attend = packer(CacheBatch), packer(CacheAppendArgs), packer(CacheAttendArgs)
_INT_MAX = 2 ** 31 - 1


class PagedCache:
    """Keys and values of many sequences in pages of ``page_size`` positions:
    ``k_pages`` and ``v_pages`` are contiguous [num_pages, Hkv, page_size, D] (bf16 or fp32,
    on one GPU), and position t of sequence b lies in page ``block_table[b, t // page_size]``.

    The new tokens of a call are packed along the first axis of [T, heads, D] tensors:
    ``cu_tokens`` int32 [B + 1] gives each sequence's rows (None: T / B rows each), and
    ``seq_lens`` int32 [B] the sequences' lengths with the new tokens.  ``block_table`` is
    int32 [B, max_pages].  These stay on the device and are not read by the host: a page or
    position that does not exist is left out, and ``check()`` reports it.

    ``k_pages`` and ``v_pages`` stay the tensors that the cache was made of."""

    def __init__(self, k_pages: torch.Tensor, v_pages: torch.Tensor):
        self._lib = load_library()
        if k_pages.dim() != 4 or k_pages.shape != v_pages.shape:
            raise ValueError("k_pages and v_pages must be [num_pages, Hkv, page_size, D] of one shape")
        if k_pages.dtype != v_pages.dtype:
            raise TypeError("k_pages and v_pages must have one dtype")
        if not k_pages.is_cuda or k_pages.device != v_pages.device:
            raise ValueError("k_pages and v_pages must be CUDA tensors on one device")
        if not k_pages.is_contiguous() or not v_pages.is_contiguous():
            raise ValueError("k_pages and v_pages must be contiguous")
        pages, self.num_kv_heads, self.page_size, self.head_dim = k_pages.shape
        if self.head_dim not in (64, 128) or self.page_size % 16 or min(pages, self.num_kv_heads, self.page_size) < 1:
            raise ValueError("a cache needs pages and heads, a head_dim of 64 or 128 and a page_size that is a "
                             f"multiple of 16, got {tuple(k_pages.shape)}")
        self._k_pages, self._v_pages, self.dtype = k_pages, v_pages, k_pages.dtype
        self._error = torch.zeros(1, dtype=torch.int32, device=k_pages.device)
        self._at = k_pages.data_ptr(), v_pages.data_ptr()
        self._cache = Cache(*self._at, pages, self.num_kv_heads, self.page_size, self.head_dim,
                            _dtype_code(self.dtype), self._error.data_ptr())
        self._ref = bytes(self._cache)
        self._device = k_pages.device

    @property
    def k_pages(self) -> torch.Tensor:
        return self._k_pages

    @property
    def v_pages(self) -> torch.Tensor:
        return self._v_pages

    def _enter(self, stream):
        # the library holds the pages' addresses
        if (self._k_pages.data_ptr(), self._v_pages.data_ptr()) != self._at:
            raise ValueError("the pages have moved in memory; make a new PagedCache of them")
        return elsewhere(self._k_pages, "k_pages", stream)

    def _rows(self, t, name, T=None, heads=None):
        strides = check_rows(t, name, self._device, 3, self.dtype)
        n, h, d = t.shape
        if d != self.head_dim or (T is not None and n != T) or (heads is not None and h != heads):
            raise ValueError(f"{name} must be [{'T' if T is None else T}, {'heads' if heads is None else heads}, "
                             f"{self.head_dim}], got {tuple(t.shape)}")
        return strides

    def _batch(self, T, seq_lens, block_table, cu_tokens) -> bytes:
        B = seq_lens.shape[0]
        if block_table.dim() != 2 or block_table.shape[0] != B or block_table.shape[1] < 1:
            raise ValueError(f"block_table must be [{B}, max_pages], got {tuple(block_table.shape)}")
        if cu_tokens is None and (T or B) and (B == 0 or T % B):
            raise ValueError(f"{T} rows cannot be shared by {B} sequences; pass cu_tokens")
        device = self._device
        return _pack_batch(B, T, check_index(block_table, "block_table", device, block_table.shape),
                           block_table.shape[1], check_index(seq_lens, "seq_lens", device, (B,)),
                           check_index(cu_tokens, "cu_tokens", device, (B + 1,)))

    def append(self, k: torch.Tensor, v: torch.Tensor, seq_lens: torch.Tensor, block_table: torch.Tensor, *,
               q: Optional[torch.Tensor] = None, cu_tokens: Optional[torch.Tensor] = None,
               rotary: Optional[Rotary] = None, norm_eps: Optional[float] = None,
               q_weight: Optional[torch.Tensor] = None, k_weight: Optional[torch.Tensor] = None,
               q_out: Optional[torch.Tensor] = None, stream=None) -> Optional[torch.Tensor]:
        """Write the new tokens' k and v [T, Hkv, D] (any strides with a dense last axis) into
        the pages, k normed (``norm_eps``, as in ``Rotary.forward``) and rotated at its
        position; q [T, Hq, D] is normed and rotated alike into ``q_out``, which is returned
        (it may be q; rows of no sequence are not written)."""
        ctx = self._enter(stream)
        if ctx is None:
            return self._append(k, v, seq_lens, block_table, q, cu_tokens, rotary, norm_eps, q_weight, k_weight, q_out)
        with ctx:
            return self._append(k, v, seq_lens, block_table, q, cu_tokens, rotary, norm_eps, q_weight, k_weight, q_out)

    def _append(self, k, v, seq_lens, block_table, q, cu_tokens, rotary, norm_eps, q_weight, k_weight, q_out):
        ks = self._rows(k, "k", heads=self.num_kv_heads)
        T = k.shape[0]
        vs = self._rows(v, "v", T, self.num_kv_heads)
        if rotary is not None and rotary.head_dim != self.head_dim:
            raise ValueError(f"the rotation is for head_dim {rotary.head_dim}, the cache's is {self.head_dim}")
        Hq, qs, os, q_ptr, qo_ptr = 0, (0, 0), (0, 0), 0, 0
        if q is None:
            q_out = None
        else:
            qs = self._rows(q, "q", T)
            Hq = q.shape[1]
            if q_out is None:
                q_out = torch.empty_like(q, memory_format=torch.contiguous_format)
                os = (Hq * self.head_dim, self.head_dim)
            else:
                os = self._rows(q_out, "q_out", T, Hq)
            q_ptr, qo_ptr = q.data_ptr(), q_out.data_ptr()
        batch = self._batch(T, seq_lens, block_table, cu_tokens)
        a = _pack_append(
            Hq, q_ptr, k.data_ptr(), v.data_ptr(), qs[0], qs[1], ks[0], ks[1], vs[0], vs[1], qo_ptr, os[0], os[1],
            *(NO_ROTATION if rotary is None else rotary.fields),
            *head_norm(norm_eps, q_weight, k_weight, self.head_dim, self._device))
        st = self._lib.swa_cache_append(self._ref, batch, a, current_stream(self._k_pages))
        if st != 0:
            raise SwaError(st, "swa_cache_append")
        return q_out

    def attend(self, q: torch.Tensor, seq_lens: torch.Tensor, block_table: torch.Tensor, *,
               cu_tokens: Optional[torch.Tensor] = None, max_tokens: Optional[int] = None, max_len: int = 0,
               window: Optional[int] = None, softcap: float = 0.0, scale: float = 0.0,
               out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None, return_lse: bool = True,
               stream=None):
        """Attention of the new tokens' q [T, Hq, D] over their sequences' keys (their own
        included): each token sees the positions up to its own, the last ``window`` ones
        before it only when that is given.  With ``cu_tokens``, ``max_tokens`` bounds a
        sequence's new tokens (T when None); ``max_len`` bounds ``seq_lens`` (0: the table's
        capacity).  One window serves all heads, and there is no dilation.  ``softcap`` c > 0
        turns a score s into ``c tanh(s / c)``; scale 0 is 1/sqrt(D).  Returns ``(out, lse)``:
        [T, Hq, D] and fp32 [T, Hq] (natural log); rows of no sequence are not written."""
        ctx = self._enter(stream)
        args = (q, seq_lens, block_table, cu_tokens, max_tokens, max_len, window, softcap, scale, out, lse, return_lse)
        if ctx is None:
            return self._attend(*args)
        with ctx:
            return self._attend(*args)

    def _attend(self, q, seq_lens, block_table, cu_tokens, max_tokens, max_len, window, softcap, scale, out, lse,
                return_lse):
        qs = self._rows(q, "q")
        T, Hq, D = q.shape
        if window is None:
            window = -1
        elif window < 0:
            raise ValueError("window must be None or at least 0")
        check_fp32(softcap, "softcap")
        check_fp32(scale, "scale")
        # bounds beyond what an int32 length can reach bound nothing
        window = min(window, _INT_MAX)
        max_len = min(max_len, _INT_MAX)
        max_tokens = T if max_tokens is None else min(max_tokens, T)
        batch = self._batch(T, seq_lens, block_table, cu_tokens)
        if out is None:
            out = torch.empty_like(q, memory_format=torch.contiguous_format)
        else:
            self._rows(out, "out", T, Hq)
            if not out.is_contiguous():
                raise ValueError("out must be contiguous")
        if lse is None:
            if return_lse:
                lse = q.new_empty((T, Hq), dtype=torch.float32)
        elif lse.dtype != torch.float32 or lse.shape != (T, Hq) or not lse.is_contiguous() or \
                lse.device != self._device:
            raise ValueError(f"lse must be a contiguous fp32 [{T}, {Hq}] on {self._device}")
        fields = (Hq, q.data_ptr(), qs[0], qs[1], max_tokens, max_len, window, softcap, scale, out.data_ptr(),
                  0 if lse is None else lse.data_ptr())
        a = _pack_attend(*fields, 0, 0)
        need = self._lib.swa_cache_attend_workspace_bytes(self._ref, batch, a)
        if need:
            ws = torch.empty(need, dtype=torch.uint8, device=self._device)
            a = _pack_attend(*fields, ws.data_ptr(), need)
        st = self._lib.swa_cache_attend(self._ref, batch, a, current_stream(self._k_pages))
        if st != 0:
            raise SwaError(st, "swa_cache_attend")
        return out, lse

    def check(self, stream=None) -> int:
        """Synchronise, read and clear the cache's error word (0 = OK)."""
        ctx = elsewhere(self._k_pages, "k_pages", stream)
        if ctx is None:
            return int(self._lib.swa_cache_check(self._ref, current_stream(self._k_pages)))
        with ctx:
            return int(self._lib.swa_cache_check(self._ref, current_stream(self._k_pages)))
