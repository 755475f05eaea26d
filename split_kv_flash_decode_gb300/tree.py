"""Convenience layer over fd_tree_decode, fd_tree_verify and fd_tree_keep: a step of speculative decoding.

Shapes, types and devices are checked here (the C ABI sees only pointers); every byte of compute
happens in the library's kernels.
"""
from __future__ import annotations

import torch

from . import _binding as B
from .decode import _KV_DTYPE, _TORCH_DTYPE, cache_shape, empty, launch, stream_address
from .rows import CacheCalls


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
        self._workspace_bytes = self.info["workspace_bytes"]
        self._t16, self._kv = _TORCH_DTYPE[self.dtype], _KV_DTYPE[self.dtype]
        self._decode, self._verify, self._keep = B.lib().fd_tree_decode, B.lib().fd_tree_verify, B.lib().fd_tree_keep
        self._q_shape, self._lse_shape = (self.tokens, self.Hq, self.d), (self.tokens, self.Hq)
        self._path_shape = (self.Bsz, self.max_drafts)
        self._cache_shape = cache_shape(self.dtype, self.Hkv, self.d, self.seqlens, 0, self.page_size)
        self._like = {}

    def _launch(self, name, call, args, stream):
        index = self.device.index
        rc = launch(index, stream_address(index, stream), call, self.tree.handle, *args)
        if rc != B.FD_OK:
            raise B.FdError(rc, name)

    def _out(self, name, t, shape, dtype, stream):
        """(tensor, address) of an output, allocated if missing."""
        if t is not None:
            return t, self._whole(name, t, shape, dtype)
        if stream is None:
            # Like one of its shape and type that is kept for this: half of torch.empty's time.
            like = self._like.get(name)
            if like is None:
                like = self._like[name] = torch.empty(shape, dtype=dtype, device=self.device)
            t = torch.empty_like(like)
        else:
            t = empty(stream, shape, dtype, self.device)
        return t, t.data_ptr()

    def __call__(self, q, k_cache, v_cache, mask=None, *, block_table=None, out=None, lse=None, status=None,
                 stream=None):
        """(out, lse) of the drafted tokens: q and out [T, Hq, d], lse [T, Hq].

        mask: int64 [T], bit j of a token's mask set where it sees node j of its sequence (tree_masks);
        None: each token sees itself and the nodes before it.
        """
        q_ptr = self._whole("q", q, self._q_shape, self._t16)
        k, v, num_pages, table, stride = self._caches(k_cache, v_cache, block_table)
        bits = 0 if mask is None else self._whole("mask", mask, (self.tokens,), torch.int64)
        out, out_ptr = self._out("out", out, self._q_shape, self._t16, stream)
        lse, lse_ptr = self._out("lse", lse, self._lse_shape, torch.float32, stream)
        state = self._status(status)
        if self.tokens:  # no tokens: empty tensors have null addresses
            work, work_ptr = None, 0
            if self._workspace_bytes:
                # Of its stream's pool, and of this call alone: another call in flight cannot meet it.
                work = torch.empty(self._workspace_bytes, dtype=torch.uint8, device=self.device) if stream is None else \
                    empty(stream, (self._workspace_bytes,), torch.uint8, self.device)
                work_ptr = work.data_ptr()
            self._launch("fd_tree_decode", self._decode,
                         (q_ptr, k, v, num_pages, table, stride, bits, out_ptr, lse_ptr, work_ptr, state), stream)
        return out, lse

    def _rows_of(self, name, t, vocab):
        """(address, row stride) of probabilities."""
        if t.dtype != torch.float32 or t.shape != (self.tokens, vocab) or t.device != self.device:
            self._refuse(name, t, (self.tokens, vocab), torch.float32)
        if vocab > 1 and t.stride(1) != 1:
            raise ValueError(f"the elements of a row of {name} must be contiguous")
        return t.data_ptr(), t.stride(0) if self.tokens > 1 else vocab

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
        tok = self._whole("tokens", tokens, (self.tokens,), torch.int32)
        u = self._whole("uniform", uniform, (self.tokens,), torch.float32)
        up = 0 if parents is None else self._whole("parents", parents, (self.tokens,), torch.int32)
        path, path_ptr = self._out("path", path, self._path_shape, torch.int32, stream)
        emitted, emitted_ptr = self._out("emitted", emitted, self._path_shape, torch.int32, stream)
        count, count_ptr = self._out("count", count, (self.Bsz,), torch.int32, stream)
        self._launch("fd_tree_verify", self._verify,
                     (p, p_stride, d, d_stride, vocab, tok, up, u, path_ptr, emitted_ptr, count_ptr), stream)
        return path, emitted, count

    def keep(self, k_cache, v_cache, path, count, *, block_table=None, status=None, stream=None):
        """Moves the rows of path's nodes to the front of the drafted ones, in place."""
        k, v, num_pages, table, stride = self._caches(k_cache, v_cache, block_table)
        way = self._whole("path", path, self._path_shape, torch.int32)
        many = self._whole("count", count, (self.Bsz,), torch.int32)
        state = self._status(status)
        if self.tokens:
            self._launch("fd_tree_keep", self._keep,
                         (k, v, num_pages, table, stride, way, self.max_drafts, many, state), stream)
