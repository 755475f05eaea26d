"""Convenience layer over fd_append and fd_gather: what writes and reads back a KV cache.

Shapes, types and devices are checked here (the C ABI sees only pointers); every byte of
compute happens in the library's kernels.
"""
from __future__ import annotations

import ctypes

import torch

from . import _binding as B
from .decode import _KV_DTYPE, _TORCH_DTYPE, cache_shape


class Rope:
    """A rotary embedding: one frequency (radians per position) per rotated pair.

    ``inv_freq`` has rot_dim / 2 entries, which may carry any scaling of long contexts.  ``axes``
    gives the position axis of each pair (images and video: time, height, width), ``scale`` is a
    factor on cos and sin.  Pairs are (i, i + rot_dim / 2), or (2 i, 2 i + 1) if ``interleaved``.
    """

    def __init__(self, inv_freq, interleaved=False, axes=None, scale=1.0):
        freq = [float(x) for x in inv_freq]
        n = len(freq)
        self._freq = (ctypes.c_double * max(1, n))(*freq)
        self._axis = None
        self.num_axes = 1
        if axes is not None:
            axes = [int(x) for x in axes]
            if len(axes) != n or any(not 0 <= x <= 255 for x in axes):
                raise ValueError("axes needs one small non-negative integer per frequency")
            self._axis = (ctypes.c_uint8 * max(1, n))(*axes)
            self.num_axes = max(axes, default=0) + 1
        self.rot_dim = 2 * n
        self.args = B.RopeArgs(rot_dim=self.rot_dim, interleaved=int(bool(interleaved)),
                               inv_freq=ctypes.addressof(self._freq),
                               axis=ctypes.addressof(self._axis) if self._axis else None,
                               num_axes=self.num_axes, scale=float(scale))


class KVRows:
    """The rows [begin_b, begin_b + count_b) of every sequence of a cache (default: all rows).

    ``seqlens`` are the lengths the cache is laid out for, the rows of the call included: the
    ones a Decoder of the same cache takes.  Owns host memory only.
    """

    def __init__(self, Hq, Hkv, d, seqlens, begin=None, count=None, dtype="f16", page_size=0,
                 device=None):
        dev = torch.device(device if device is not None else "cuda")
        if dev.type != "cuda":
            raise ValueError("KVRows needs a CUDA device")
        self.device = torch.device("cuda", dev.index if dev.index is not None
                                   else torch.cuda.current_device())
        self.seqlens = [int(x) for x in seqlens]
        self.Bsz = len(self.seqlens)
        self.Hq, self.Hkv, self.d, self.dtype = int(Hq), int(Hkv), int(d), dtype
        self.page_size = int(page_size)
        begin = [0] * self.Bsz if begin is None else [int(x) for x in begin]
        if count is None:
            count = [n - a for n, a in zip(self.seqlens, begin)]
        self.rows = B.fd_rows_plan(self.Bsz, self.Hq, self.Hkv, self.d, self.seqlens, begin, count,
                                   self.page_size, dtype)
        self.tokens = self.rows.tokens
        self._cache_shape = None if self.page_size else cache_shape(dtype, self.Hkv, self.d, self.seqlens)

    def _tensor(self, name, t, shape, dtype):
        if t.dtype != dtype or t.device != self.device or tuple(t.shape) != shape:
            raise ValueError(f"{name} is {t.dtype} {tuple(t.shape)} on {t.device}, expected "
                             f"{dtype} {shape} on {self.device}")
        return t

    def _whole(self, name, t, shape, dtype):
        if not self._tensor(name, t, shape, dtype).is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        return t.data_ptr()

    def _input(self, name, t, heads):
        self._tensor(name, t, (self.tokens, heads, self.d), _TORCH_DTYPE[self.dtype])
        a, b, c = t.stride()
        if c != 1 and t.numel() > 0:
            raise ValueError(f"the elements of a head of {name} must be contiguous")
        # A dimension of size 1 is never stepped along, whatever stride it reports.
        return t.data_ptr(), (a if self.tokens > 1 else 0, b if heads > 1 else 0)

    def _caches(self, k_cache, v_cache, block_table):
        num_pages, stride, table = 0, 0, None
        shape = self._cache_shape
        if self.page_size:
            if block_table is None:
                raise ValueError("a paged cache needs its block_table")
            num_pages = k_cache.shape[0]
            shape = cache_shape(self.dtype, self.Hkv, self.d, None, num_pages, self.page_size)
            stride = block_table.shape[1] if block_table.dim() == 2 else -1
            table = self._whole("block_table", block_table, (self.Bsz, stride), torch.int32)
        elif block_table is not None:
            raise ValueError("these rows are of a contiguous cache")
        kv = _KV_DTYPE[self.dtype]
        return (self._whole("k_cache", k_cache, shape, kv), self._whole("v_cache", v_cache, shape, kv),
                num_pages, table, stride)

    def _status(self, status):
        return None if status is None else self._whole("status", status, (1,), torch.int32)

    def append(self, q=None, k=None, v=None, k_cache=None, v_cache=None, *, q_norm=None, k_norm=None,
               q_weight=None, k_weight=None, eps=1e-6, weight_offset=0.0, rope=None, positions=None,
               block_table=None, q_out=None, k_out=None, k_mul=1.0, v_mul=1.0, status=None,
               stream=None):
        """Norm and rotate q and k, store k and v in the cache; returns q_out (None without q).

        q [T, Hq, d], k and v [T, Hkv, d] in any strides with whole heads; T tokens in the order
        of the rows.  A head is normalised where its weight (or q_norm / k_norm) is given.
        positions: int32 [T], or [axes, T]; default: each token's row.  q_out and k_out
        [T, heads, d] contiguous (or q and k themselves); q_out is allocated if missing.
        """
        a = B.AppendArgs()
        t16 = _TORCH_DTYPE[self.dtype]
        if q is not None:
            a.q, a.q_stride[:] = self._input("q", q, self.Hq)
            if q_out is None:
                q_out = torch.empty((self.tokens, self.Hq, self.d), dtype=t16, device=self.device)
            a.q_out = self._whole("q_out", q_out, (self.tokens, self.Hq, self.d), t16)
        elif q_out is not None:
            raise ValueError("q_out without q")
        if k is not None:
            a.k, a.k_stride[:] = self._input("k", k, self.Hkv)
        if v is not None:
            a.v, a.v_stride[:] = self._input("v", v, self.Hkv)
        if k_out is not None:
            a.k_out = self._whole("k_out", k_out, (self.tokens, self.Hkv, self.d), t16)
        if (k_cache is None) != (v_cache is None):
            raise ValueError("k_cache and v_cache come together")
        if k_cache is not None:
            a.k_cache, a.v_cache, a.num_pages, a.block_table, a.bt_stride = \
                self._caches(k_cache, v_cache, block_table)
        for name, w, heads in (("q_weight", q_weight, q), ("k_weight", k_weight, k)):
            if w is not None:
                if heads is None:
                    raise ValueError(f"{name} without its input")
                setattr(a, name, self._whole(name, w, (self.d,), t16))
        a.q_norm = int(q_weight is not None if q_norm is None else q_norm)
        a.k_norm = int(k_weight is not None if k_norm is None else k_norm)
        a.eps, a.weight_offset = eps, weight_offset
        a.k_mul, a.v_mul = k_mul, v_mul
        if rope is not None:
            a.rope = ctypes.addressof(rope.args)
            if positions is not None:
                if positions.dim() == 1 and rope.num_axes == 1:
                    shape, a.pos_stride = (self.tokens,), self.tokens
                else:
                    shape, a.pos_stride = (rope.num_axes, self.tokens), self.tokens
                a.positions = self._whole("positions", positions, shape, torch.int32)
        elif positions is not None:
            raise ValueError("positions without rope")
        a.status = self._status(status)
        if self.tokens:  # no rows: empty tensors have null addresses
            self._on_device(B.fd_append, self.rows, a, stream)
        return q_out

    def gather(self, k_cache, v_cache, *, block_table=None, k_out=None, v_out=None, status=None,
               stream=None):
        """The rows of K and V back in 16 bits: (k, v), each [T, Hkv, d]."""
        k_ptr, v_ptr, num_pages, table, stride = self._caches(k_cache, v_cache, block_table)
        shape, t16 = (self.tokens, self.Hkv, self.d), _TORCH_DTYPE[self.dtype]
        k_out = torch.empty(shape, dtype=t16, device=self.device) if k_out is None else k_out
        v_out = torch.empty(shape, dtype=t16, device=self.device) if v_out is None else v_out
        k_to, v_to = self._whole("k_out", k_out, shape, t16), self._whole("v_out", v_out, shape, t16)
        if self.tokens:
            self._on_device(B.fd_gather, self.rows, k_ptr, v_ptr, num_pages, table, stride, k_to, v_to,
                            self._status(status), stream)
        return k_out, v_out

    def _on_device(self, call, *args):
        if torch.cuda.current_device() == self.device.index:
            call(*args)
        else:
            with torch.cuda.device(self.device):
                call(*args)
