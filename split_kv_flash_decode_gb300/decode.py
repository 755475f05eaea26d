"""Convenience layer over the C ABI: a Decoder owns a plan and its workspace.

Shapes and dtypes are checked here (the C ABI sees only pointers); every byte
of compute happens in fd_decode's kernel.
"""
from __future__ import annotations

import contextlib

import torch

from . import _binding as B

# q / out type and K / V storage type of each plan dtype.
_TORCH_DTYPE = {"f16": torch.float16, "bf16": torch.bfloat16, "f16_e4m3kv": torch.float16,
                "f16_e2m1kv": torch.float16, "bf16_e2m1kv": torch.bfloat16}
_KV_DTYPE = {"f16": torch.float16, "bf16": torch.bfloat16, "f16_e4m3kv": torch.uint8,
             "f16_e2m1kv": torch.uint8, "bf16_e2m1kv": torch.uint8}


# torch's current device and stream without the Python objects around them (a tenth of their cost).
_device_now = getattr(torch._C, "_cuda_getDevice", None)  # missing in builds without CUDA
_stream_now = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def stream_address(index, stream):
    """Raw stream of an address or of anything with a cuda_stream; None is the current stream of device `index`."""
    return _stream_now(index) if stream is None else B._stream(stream)


def launch(index, address, call, *args):
    """call(*args, address) with device `index` current."""
    if _device_now() == index:
        return call(*args, address)
    with torch.cuda.device(index):
        return call(*args, address)


def on_stream(stream, device):
    """Context in which allocations come from the pool of `stream` (None: the current one), in whose
    order they are used: memory just freed on another stream may still be in use there."""
    if stream is None:
        return contextlib.nullcontext()
    if not isinstance(stream, torch.cuda.Stream):
        address = B._stream(stream)
        # 1 is the runtime's handle of the default stream, which torch would read as an id of its own.
        stream = torch.cuda.ExternalStream(address, device) if address > 1 else torch.cuda.default_stream(device)
    return torch.cuda.stream(stream)


def empty(stream, shape, dtype, device):
    """torch.empty from the pool of the stream that will write it."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with on_stream(stream, device):
        return torch.empty(shape, dtype=dtype, device=device)


def cache_shape(dtype, Hkv, d, seqlens=None, num_pages=None, page_size=0):
    """Shape of the K (and of the V) cache: of the contiguous cache of `seqlens`, or of a pool of
    `num_pages` pages.  4-bit caches are made of blocks of 16 tokens (include/fd.h)."""
    unit, last = (16, 9 * d) if str(dtype).endswith("e2m1kv") else (1, d)
    if page_size:
        return (num_pages, page_size // unit, Hkv, last)
    return (sum((int(x) + unit - 1) // unit for x in seqlens), Hkv, last)


class Decoder:
    """Plan and zeroed workspaces for one decode shape on one device.

    Every stream that a call runs on has a workspace of its own, allocated and zeroed in that
    stream's order (``workspace`` is the one of the stream that was current at construction).  A
    captured call allocates none: it takes its stream's, or else the first, whose zeroing has to be
    over when the capture begins (torch.cuda.graph waits for it).  Replays of such graphs, and calls
    on the streams whose workspace they took, must not overlap, and the Decoder outlives the graphs.
    """

    def __init__(self, Hq, Hkv, d, seqlens, W, dtype="f16", flags=0, chunks=0, device=None,
                 num_sms=0, page_size=0):
        dev = torch.device(device if device is not None else "cuda")
        if dev.type != "cuda":
            raise ValueError("Decoder needs a CUDA device")
        self.device = torch.device("cuda", dev.index if dev.index is not None
                                   else torch.cuda.current_device())
        self.seqlens = [int(x) for x in seqlens]
        self.Bsz = len(self.seqlens)
        self.Hq, self.Hkv, self.d, self.dtype = int(Hq), int(Hkv), int(d), dtype
        self.n_tokens = sum(self.seqlens)
        self.page_size = int(page_size)
        with torch.cuda.device(self.device):
            if self.page_size:
                self.plan = B.fd_plan_paged(self.Bsz, Hq, Hkv, d, self.seqlens, W, self.page_size,
                                            dtype, flags, chunks, num_sms)
            else:
                self.plan = B.fd_plan(self.Bsz, Hq, Hkv, d, self.seqlens, W, dtype, flags, chunks,
                                      num_sms)
            self.workspace = self._zeros()
            self._home = stream_address(self.device.index, None)
        self._others = {}  # workspaces of other streams, by address
        self._shapes()

    def _zeros(self):
        return torch.zeros(max(1, self.plan.workspace_bytes), dtype=torch.uint8, device=self.device)

    def _workspace(self, address):
        """The workspace of the stream at this address."""
        if address == self._home:
            return self.workspace
        ws = self._others.get(address)
        if ws is None:
            with on_stream(address, self.device):
                if torch.cuda.is_current_stream_capturing():
                    return self.workspace
                ws = self._others[address] = self._zeros()
        return ws

    def _shapes(self):
        """What every call compares its tensors with."""
        dtype = self.dtype
        self._q_shape, self._lse_shape = (self.Bsz, self.Hq, self.d), (self.Bsz, self.Hq)
        self._t16, self._kv = _TORCH_DTYPE.get(dtype), _KV_DTYPE.get(dtype)
        self._decode, self._decode_paged = B.lib().fd_decode, B.lib().fd_decode_paged
        self._kv_shape = cache_shape(dtype, self.Hkv, self.d, self.seqlens)
        self._page_shape = cache_shape(dtype, self.Hkv, self.d, None, 0, self.page_size or 16)[1:]

    @property
    def info(self) -> dict:
        return self.plan.info

    def _refuse(self, name, t, shape, dtype):
        if t.device != self.device:
            raise ValueError(f"{name} is on {t.device}, expected {self.device}")
        if t.dtype != dtype:
            raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")
        if t.shape != shape:
            raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
        raise ValueError(f"{name} must be contiguous")

    def _check(self, name, t, shape, dtype):
        """Address of a contiguous tensor of this shape and type on the device."""
        if t.shape != shape or t.dtype != dtype or t.device != self.device or not t.is_contiguous():
            self._refuse(name, t, shape, dtype)
        return t.data_ptr()

    def _run(self, call, name, q, kv, out, lse, stream):
        """call(plan, q, *kv, out, lse, workspace, stream), out and lse allocated where missing."""
        q_ptr = self._check("q", q, self._q_shape, self._t16)
        if out is None:
            out = empty(stream, self._q_shape, self._t16, self.device)
            out_ptr = out.data_ptr()
        else:
            out_ptr = self._check("out", out, self._q_shape, self._t16)
        if lse is None:
            lse = empty(stream, self._lse_shape, torch.float32, self.device)
            lse_ptr = lse.data_ptr()
        else:
            lse_ptr = self._check("lse", lse, self._lse_shape, torch.float32)
        index = self.device.index
        address = stream_address(index, stream)
        rc = launch(index, address, call, self.plan.handle, q_ptr, *kv, out_ptr, lse_ptr,
                    self._workspace(address).data_ptr())
        if rc != B.FD_OK:
            raise B.FdError(rc, name)
        return out, lse

    def __call__(self, q, k, v, out=None, lse=None, stream=None):
        kv = (self._check("k", k, self._kv_shape, self._kv), self._check("v", v, self._kv_shape, self._kv))
        return self._run(self._decode, "fd_decode", q, kv, out, lse, stream)

    def decode_paged(self, q, k_pages, v_pages, block_table, out=None, lse=None, stream=None):
        """Decode over a paged cache: pools [num_pages, page_size, Hkv, d] (or as cache_shape says),
        int32 block_table [B, stride]."""
        if not self.page_size:
            raise ValueError("this Decoder was planned for contiguous K/V")
        num_pages = k_pages.shape[0]
        shape = (num_pages, *self._page_shape)
        if block_table.dtype != torch.int32 or block_table.dim() != 2 or \
                block_table.shape[0] != self.Bsz or not block_table.is_contiguous() or \
                block_table.device != self.device:
            raise ValueError("block_table must be a contiguous int32 [B, stride] tensor on the device")
        kv = (self._check("k_pages", k_pages, shape, self._kv), self._check("v_pages", v_pages, shape, self._kv),
              num_pages, block_table.data_ptr(), block_table.shape[1])
        return self._run(self._decode_paged, "fd_decode_paged", q, kv, out, lse, stream)

    def status(self, stream=None) -> int:
        """fd_workspace_status of this Decoder's decodes: synchronises `stream` (None: the current
        one), or the device where calls ran on several streams."""
        with torch.cuda.device(self.device):
            if self._others:
                torch.cuda.synchronize()
            found = [B.fd_workspace_status(self.plan, ws, stream) for ws in (self.workspace, *self._others.values())]
        return next((x for x in found if x != B.FD_OK), B.FD_OK)


def flash_decode(q, k, v, seqlens, W, flags=0, chunks=0):
    """One-shot decode: plan, allocate, run.  Returns (out, lse)."""
    dtype = {torch.float16: "f16", torch.bfloat16: "bf16"}[q.dtype]
    if k.dtype == torch.uint8:
        dtype = dtype + "_e2m1kv" if k.shape[2] == 9 * q.shape[2] else "f16_e4m3kv"
    dec = Decoder(q.shape[1], k.shape[1], q.shape[2], seqlens, W, dtype, flags, chunks,
                  device=q.device)
    return dec(q, k, v)
