"""Convenience layer over fd_append and fd_gather: what writes and reads back a KV cache.

Shapes, types and devices are checked here (the C ABI sees only pointers); every byte of
compute happens in the library's kernels.
"""
from __future__ import annotations

import ctypes

import torch

from . import _binding as B
from .decode import _KV_DTYPE, _TORCH_DTYPE, cache_shape, empty, launch, stream_address


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
        self.address = ctypes.addressof(self.args)


class CacheCalls:
    """Argument checks of calls on a cache: of KVRows, and of TreeDecoder.

    Uses device, Bsz, page_size, _kv and _cache_shape (of a paged cache: with any number of pages)."""

    def _refuse(self, name, t, shape, dtype):
        raise ValueError(f"{name} is {t.dtype} {tuple(t.shape)} (strides {t.stride()}) on {t.device}, expected "
                         f"a contiguous {dtype} {tuple(shape)} on {self.device}")

    def _whole(self, name, t, shape, dtype):
        """Address of a contiguous tensor."""
        if t.dtype != dtype or t.shape != shape or t.device != self.device or not t.is_contiguous():
            self._refuse(name, t, shape, dtype)
        return t.data_ptr()

    def _caches(self, k_cache, v_cache, block_table):
        """(k, v, num_pages, block table, its stride)."""
        num_pages, stride, table, shape = 0, 0, 0, self._cache_shape
        if self.page_size:
            if block_table is None:
                raise ValueError("a paged cache needs its block_table")
            num_pages = k_cache.shape[0]
            shape = (num_pages, *shape[1:])
            stride = block_table.shape[-1] if block_table.dim() == 2 else -1
            table = self._whole("block_table", block_table, (self.Bsz, stride), torch.int32)
        elif block_table is not None:
            raise ValueError("these rows are of a contiguous cache")
        return (self._whole("k_cache", k_cache, shape, self._kv), self._whole("v_cache", v_cache, shape, self._kv),
                num_pages, table, stride)

    def _status(self, status):
        return 0 if status is None else self._whole("status", status, (1,), torch.int32)


class KVRows(CacheCalls):
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
        self._t16, self._kv = _TORCH_DTYPE[dtype], _KV_DTYPE[dtype]
        self._append, self._gather = B.lib().fd_append, B.lib().fd_gather
        self._q_shape = (self.tokens, self.Hq, self.d)
        self._k_shape = (self.tokens, self.Hkv, self.d)
        self._cache_shape = cache_shape(dtype, self.Hkv, self.d, self.seqlens, 0, self.page_size)

    def _input(self, name, t, shape):
        """Address and strides of q, k or v (0 for a dimension of size 1: it is never stepped along)."""
        if t.dtype != self._t16 or t.shape != shape or t.device != self.device:
            self._refuse(name, t, shape, self._t16)
        a, b, c = t.stride()
        if c != 1 and shape[0] > 0:
            raise ValueError(f"the elements of a head of {name} must be contiguous")
        return t.data_ptr(), a if shape[0] > 1 else 0, b if shape[1] > 1 else 0

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
        q_in = k_in = v_in = (0, 0, 0)
        q_to = k_to = q_w = k_w = rope_ptr = pos = pos_stride = 0
        cache = (0, 0, 0, 0, 0)
        if q is not None:
            q_in = self._input("q", q, self._q_shape)
            if q_out is None:
                q_out = empty(stream, self._q_shape, self._t16, self.device)
                q_to = q_out.data_ptr()
            else:
                q_to = self._whole("q_out", q_out, self._q_shape, self._t16)
        elif q_out is not None:
            raise ValueError("q_out without q")
        if k is not None:
            k_in = self._input("k", k, self._k_shape)
        if v is not None:
            v_in = self._input("v", v, self._k_shape)
        if k_out is not None:
            k_to = self._whole("k_out", k_out, self._k_shape, self._t16)
        if (k_cache is None) != (v_cache is None):
            raise ValueError("k_cache and v_cache come together")
        if k_cache is not None:
            cache = self._caches(k_cache, v_cache, block_table)
        if q_weight is not None:
            if q is None:
                raise ValueError("q_weight without q")
            q_w = self._whole("q_weight", q_weight, (self.d,), self._t16)
        if k_weight is not None:
            if k is None:
                raise ValueError("k_weight without k")
            k_w = self._whole("k_weight", k_weight, (self.d,), self._t16)
        if rope is not None:
            rope_ptr = rope.address
            if positions is not None:
                shape = (self.tokens,) if positions.dim() == 1 and rope.num_axes == 1 else (rope.num_axes, self.tokens)
                pos, pos_stride = self._whole("positions", positions, shape, torch.int32), self.tokens
        elif positions is not None:
            raise ValueError("positions without rope")
        args = B.APPEND_ARGS.pack(
            q_in[0], k_in[0], v_in[0], q_in[1], q_in[2], k_in[1], k_in[2], v_in[1], v_in[2],
            q_w != 0 if q_norm is None else bool(q_norm), k_w != 0 if k_norm is None else bool(k_norm),
            q_w, k_w, eps, weight_offset, rope_ptr, pos, pos_stride, q_to, k_to, cache[0], cache[1],
            k_mul, v_mul, cache[2], cache[4], cache[3], self._status(status))
        if self.tokens:  # no rows: empty tensors have null addresses
            index = self.device.index
            rc = launch(index, stream_address(index, stream), self._append, self.rows.handle, args)
            if rc != B.FD_OK:
                raise B.FdError(rc, "fd_append")
        return q_out

    def gather(self, k_cache, v_cache, *, block_table=None, k_out=None, v_out=None, status=None,
               stream=None):
        """The rows of K and V back in 16 bits: (k, v), each [T, Hkv, d]."""
        cache = self._caches(k_cache, v_cache, block_table)
        if k_out is None:
            k_out = empty(stream, self._k_shape, self._t16, self.device)
            k_to = k_out.data_ptr()
        else:
            k_to = self._whole("k_out", k_out, self._k_shape, self._t16)
        if v_out is None:
            v_out = empty(stream, self._k_shape, self._t16, self.device)
            v_to = v_out.data_ptr()
        else:
            v_to = self._whole("v_out", v_out, self._k_shape, self._t16)
        if self.tokens:
            index = self.device.index
            rc = launch(index, stream_address(index, stream), self._gather, self.rows.handle, *cache, k_to, v_to,
                        self._status(status))
            if rc != B.FD_OK:
                raise B.FdError(rc, "fd_gather")
        return k_out, v_out
