"""Convenience layer over fd_tree_decode, fd_tree_verify and fd_tree_keep: a step of speculative decoding.

Shapes, types and devices are checked here (the C ABI sees only pointers); every byte of compute
happens in the library's kernels.
"""
from __future__ import annotations

import torch

from . import _binding as B
from .decode import _KV_DTYPE, _TORCH_DTYPE, _device_now, _stream_now, cache_shape, empty, launch, stream_address
from .rows import CacheCalls

_empty_like = torch.empty_like


def tree_masks(parents):
    """(masks, depths) of one sequence's nodes: its mask has a node's own bit and those of its ancestors,
    as the signed number that an int64 tensor holds.  parents[0] is -1, parents[i] < i."""
    masks, depths = [], []
    for i, up in enumerate(parents):
        if i >= B.FD_MAX_DRAFTS or (up != -1 if i == 0 else not 0 <= up < i):
            raise ValueError("parents are -1 for the root, then of earlier nodes; at most "
                             f"{B.FD_MAX_DRAFTS} nodes")
        masks.append((masks[up] if i else 0) | 1 << i)
        depths.append(depths[up] + 1 if i else 0)
    return [x - (1 << 64) if x >> 63 else x for x in masks], depths


class TreeDecoder(CacheCalls):
    """A step over drafted tokens, the last ``drafts`` rows of every sequence of a cache.

    ``seqlens`` are the lengths the cache is laid out for, the drafted tokens included (KVRows.append
    wrote them).  Owns host memory only; workspaces come from the pool of each call's stream.
    """

    def __init__(self, Hq, Hkv, d, seqlens, drafts, dtype="f16", page_size=0, device=None, num_sms=0):
        dev = torch.device(device if device is not None else "cuda")
        if dev.type != "cuda":
            raise ValueError("TreeDecoder needs a CUDA device")
        self.device = torch.device("cuda", dev.index if dev.index is not None
                                   else torch.cuda.current_device())
        self.seqlens, self.drafts = [int(x) for x in seqlens], [int(x) for x in drafts]
        self.Bsz = len(self.seqlens)
        self.Hq, self.Hkv, self.d, self.dtype = int(Hq), int(Hkv), int(d), dtype
        self.page_size = int(page_size)
        with torch.cuda.device(self.device):
            self.tree = B.fd_tree_plan(self.Bsz, self.Hq, self.Hkv, self.d, self.seqlens, self.drafts,
                                       self.page_size, dtype, num_sms)
        self._shapes()

    def _shapes(self):
        """What every call compares its tensors with."""
        self.info = self.tree.info
        self.tokens, self.max_drafts = self.info["tokens"], self.info["max_drafts"]
        self._handle = self.tree.handle
        self._index = -1 if self.device.index is None else self.device.index  # as Tensor.get_device gives it
        self._workspace_bytes = self.info["workspace_bytes"]
        self._t16, self._kv = _TORCH_DTYPE[self.dtype], _KV_DTYPE[self.dtype]
        self._decode, self._verify, self._keep = B.lib().fd_tree_decode, B.lib().fd_tree_verify, B.lib().fd_tree_keep
        self._q_shape, self._lse_shape = (self.tokens, self.Hq, self.d), (self.tokens, self.Hq)
        self._token_shape, self._path_shape, self._count_shape = (self.tokens,), (self.Bsz, self.max_drafts), (self.Bsz,)
        self._cache_shape = cache_shape(self.dtype, self.Hkv, self.d, self.seqlens, 0, self.page_size)
        # Tensors of the outputs' shapes and types: torch.empty_like takes half of torch.empty's time.
        self._lse_like = self._path_like = self._count_like = None

    def _launch(self, name, call, args, stream):
        index = self._index
        if stream is None and _device_now() == index:
            rc = call(self._handle, *args, _stream_now(index))
        else:
            rc = launch(index, stream_address(index, stream), call, self._handle, *args)
        if rc != B.FD_OK:
            raise B.FdError(rc, name)

    def _bad(self, t, shape, dtype):
        """Whether a tensor is anything but a contiguous one of this shape and type on the device."""
        return t.dtype is not dtype or t.get_device() != self._index or t.shape != shape or not t.is_contiguous()

    def __call__(self, q, k_cache, v_cache, mask=None, *, block_table=None, out=None, lse=None, status=None,
                 stream=None):
        """(out, lse) of the drafted tokens: q and out [T, Hq, d], lse [T, Hq].

        mask: int64 [T], bit j of a token's mask set where it sees node j of its sequence (tree_masks);
        None: each token sees itself and the nodes before it.  status: an int32 word for FD_TREE_ bits; without one
        a bounded wait that gave up shows in out and lse, which are NaN there.
        """
        if self._bad(q, self._q_shape, self._t16):
            self._refuse("q", q, self._q_shape, self._t16)
        k, v, num_pages, table, stride = self._caches(k_cache, v_cache, block_table)
        if mask is not None and self._bad(mask, self._token_shape, torch.int64):
            self._refuse("mask", mask, self._token_shape, torch.int64)
        if out is None:
            out = _empty_like(q) if stream is None else empty(stream, self._q_shape, self._t16, self.device)
        elif self._bad(out, self._q_shape, self._t16):
            self._refuse("out", out, self._q_shape, self._t16)
        if lse is None:
            if stream is None:
                if self._lse_like is None:
                    self._lse_like = torch.empty(self._lse_shape, dtype=torch.float32, device=self.device)
                lse = _empty_like(self._lse_like)
            else:
                lse = empty(stream, self._lse_shape, torch.float32, self.device)
        elif self._bad(lse, self._lse_shape, torch.float32):
            self._refuse("lse", lse, self._lse_shape, torch.float32)
        state = 0 if status is None else self._status(status)
        if self.tokens:  # no tokens: empty tensors have null addresses
            work, work_ptr = None, 0
            if self._workspace_bytes:
                # Of its stream's pool, and of this call alone: another call in flight cannot meet it.
                work = torch.empty(self._workspace_bytes, dtype=torch.uint8, device=self.device) if stream is None else \
                    empty(stream, (self._workspace_bytes,), torch.uint8, self.device)
                work_ptr = work.data_ptr()
            self._launch("fd_tree_decode", self._decode,
                         (q.data_ptr(), k, v, num_pages, table, stride, 0 if mask is None else mask.data_ptr(),
                          out.data_ptr(), lse.data_ptr(), work_ptr, state), stream)
        return out, lse

    def _rows_of(self, name, t, vocab):
        """(address, row stride) of probabilities."""
        if t.dtype is not torch.float32 or t.get_device() != self._index or t.shape != (self.tokens, vocab):
            self._refuse(name, t, (self.tokens, vocab), torch.float32)
        row, one = t.stride()
        if self.tokens and vocab > 1 and one != 1:  # an empty tensor's strides say nothing
            raise ValueError(f"the elements of a row of {name} must be contiguous")
        return t.data_ptr(), row if self.tokens > 1 else vocab

    def verify(self, target, tokens, uniform, *, parents=None, draft=None, path=None, emitted=None, count=None,
               stream=None):
        """(path, emitted, count): the nodes that stand, the tokens they give and their number, of every sequence.

        target [T, V] are the target's probabilities after each token, tokens (int32) and uniform (in [0, 1))
        [T].  parents: int32 [T], each node's parent in its sequence (None: a chain).  draft [T, V]: the
        probabilities that a chain's tokens were drawn from; without it they count as given.
        path and emitted: int32 [B, max drafts], -1 behind the first count; count: int32 [B].
        """
        if target.dim() != 2 or target.shape[1] < 1:
            self._refuse("target", target, (self.tokens, "V"), torch.float32)
        vocab = target.shape[1]
        p, p_stride = self._rows_of("target", target, vocab)
        d, d_stride = (0, 0) if draft is None else self._rows_of("draft", draft, vocab)
        i32, shape = torch.int32, self._token_shape
        if self._bad(tokens, shape, i32):
            self._refuse("tokens", tokens, shape, i32)
        if self._bad(uniform, shape, torch.float32):
            self._refuse("uniform", uniform, shape, torch.float32)
        if parents is not None and self._bad(parents, shape, i32):
            self._refuse("parents", parents, shape, i32)
        if stream is None:
            if self._path_like is None:
                self._path_like = torch.empty(self._path_shape, dtype=i32, device=self.device)
                self._count_like = torch.empty(self._count_shape, dtype=i32, device=self.device)
            if path is None:
                path = _empty_like(self._path_like)
            if emitted is None:
                emitted = _empty_like(self._path_like)
            if count is None:
                count = _empty_like(self._count_like)
        else:
            path = empty(stream, self._path_shape, i32, self.device) if path is None else path
            emitted = empty(stream, self._path_shape, i32, self.device) if emitted is None else emitted
            count = empty(stream, self._count_shape, i32, self.device) if count is None else count
        for name, t, shape in (("path", path, self._path_shape), ("emitted", emitted, self._path_shape),
                               ("count", count, self._count_shape)):
            if self._bad(t, shape, i32):
                self._refuse(name, t, shape, i32)
        self._launch("fd_tree_verify", self._verify,
                     (p, p_stride, d, d_stride, vocab, tokens.data_ptr(), 0 if parents is None else parents.data_ptr(),
                      uniform.data_ptr(), path.data_ptr(), emitted.data_ptr(), count.data_ptr()), stream)
        return path, emitted, count

    def keep(self, k_cache, v_cache, path, count, *, block_table=None, status=None, stream=None):
        """Moves the rows of path's nodes to the front of the drafted ones, in place."""
        k, v, num_pages, table, stride = self._caches(k_cache, v_cache, block_table)
        if self._bad(path, self._path_shape, torch.int32):
            self._refuse("path", path, self._path_shape, torch.int32)
        if self._bad(count, self._count_shape, torch.int32):
            self._refuse("count", count, self._count_shape, torch.int32)
        state = 0 if status is None else self._status(status)
        if self.tokens:
            self._launch("fd_tree_keep", self._keep, (k, v, num_pages, table, stride, path.data_ptr(), self.max_drafts,
                                                      count.data_ptr(), state), stream)
