"""ctypes binding of libfd_gb300.so: argument marshalling only.

Every function here forwards to the C entry point of the same name in
``include/fd.h``; all compute runs in the library's CUDA kernels.  PyTorch
supplies device memory and streams.  If the library is missing the calls raise
-- there is no fallback path.
"""
from __future__ import annotations

import ctypes
import os
import struct
import threading

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_lib", "libfd_gb300.so")

FD_OK = 0
FD_ERR_INVALID = -1
FD_ERR_UNSUPPORTED = -2
FD_ERR_ALIGN = -3
FD_ERR_CUDA = -4
FD_ERR_NOMEM = -5
FD_ERR_STATE = -6
FD_ERR_TIMEOUT = -7

FD_F16 = 0
FD_BF16 = 1
FD_F16_E4M3KV = 2
FD_F16_E2M1KV = 4
FD_BF16_E2M1KV = 5
FD_PLAN_LITERAL_W = 0x1
FD_PLAN_DEBUG = 0x2
FD_PLAN_TWO_LAUNCH = 0x4
FD_PLAN_FFMA = 0x8
FD_PLAN_NO_PDL = 0x10
FD_PLAN_WAITS = 0x20
FD_PLAN_TEST_DROP_FLAG = 0x40
FD_PLAN_NO_CLUSTER = 0x80
FD_PLAN_CLUSTER = 0x100
FD_PLAN_TEST_SKIP_TILE = 0x200
FD_PLAN_TCGEN05 = 0x400
FD_PLAN_CLUSTER_COMBINE = 0x800
FD_PLAN_MMA_SYNC = 0x1000
FD_PLAN_TEST_DROP_ARRIVAL = 0x2000
FD_PLAN_DEEP_RING = 0x4000
FD_PLAN_COMBINERS_SHIFT = 16
FD_PLAN_COMBINERS_MASK = 7 << FD_PLAN_COMBINERS_SHIFT
# FD_PLAN_COMBINERS[n]: at most n CTAs share the combine of one (sequence, KV head) pair.
FD_PLAN_COMBINERS = {n: (k + 1) << FD_PLAN_COMBINERS_SHIFT for k, n in enumerate((1, 2, 4, 8, 16))}
FD_PLAN_SINGLE_COMBINER = FD_PLAN_COMBINERS[1]
FD_MAX_BATCH = 256
FD_MAX_PARTIALS = 1024
FD_MAX_DRAFTS = 64
FD_MAX_VOCAB = 1 << 20
FD_TREE_BAD_PAGE = 1
FD_TREE_BAD_PATH = 2
FD_TREE_TIMEOUT = 4

DTYPES = {"f16": FD_F16, "bf16": FD_BF16, "f16_e4m3kv": FD_F16_E4M3KV,
          "f16_e2m1kv": FD_F16_E2M1KV, "bf16_e2m1kv": FD_BF16_E2M1KV}

# Every symbol include/fd.h declares.
EXPORTED = (
    "fd_plan", "fd_plan_destroy", "fd_workspace_bytes", "fd_workspace_init", "fd_decode",
    "fd_workspace_status", "fd_strerror", "fd_plan_get_info", "fd_plan_get_range", "fd_version",
    "fd_decode_noalloc", "fd_noalloc_status", "fd_plan_paged", "fd_decode_paged",
    "fd_rows_plan", "fd_rows_destroy", "fd_rows_get_info", "fd_append", "fd_gather",
    "fd_tree_plan", "fd_tree_destroy", "fd_tree_get_info", "fd_tree_decode", "fd_tree_verify",
    "fd_tree_keep", "fd_tree_test_skip_loads",
)
FD_NOALLOC_SCRATCH_BYTES = 32 << 20


class FdError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {strerror(status)} ({status})")


class PlanInfo(ctypes.Structure):
    _fields_ = [
        ("B", ctypes.c_int32), ("Hq", ctypes.c_int32), ("Hkv", ctypes.c_int32),
        ("d", ctypes.c_int32), ("G", ctypes.c_int32), ("dtype", ctypes.c_int32),
        ("flags", ctypes.c_uint32), ("chunks", ctypes.c_int32), ("num_sms", ctypes.c_int32),
        ("ctas", ctypes.c_int32), ("max_partials", ctypes.c_int32),
        ("total_tokens", ctypes.c_int64), ("total_partials", ctypes.c_int64),
        ("workspace_bytes", ctypes.c_uint64), ("kv_bytes", ctypes.c_uint64),
        ("path", ctypes.c_int32), ("records_per_segment", ctypes.c_int32),
        ("combine_cluster", ctypes.c_int32), ("combiners", ctypes.c_int32),
        ("ctas_per_sm", ctypes.c_int32),
    ]


class RowsInfo(ctypes.Structure):
    _fields_ = [("tokens", ctypes.c_int64), ("cache_bytes", ctypes.c_int64)]


class TreeInfo(ctypes.Structure):
    _fields_ = [("tokens", ctypes.c_int64), ("max_drafts", ctypes.c_int32), ("ctas", ctypes.c_int32),
                ("workspace_bytes", ctypes.c_uint64), ("kv_bytes", ctypes.c_uint64)]


class RopeArgs(ctypes.Structure):
    """fd_rope."""
    _fields_ = [
        ("rot_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32),
        ("inv_freq", ctypes.c_void_p), ("axis", ctypes.c_void_p),
        ("num_axes", ctypes.c_int32), ("scale", ctypes.c_float),
    ]


class AppendArgs(ctypes.Structure):
    """fd_append_args."""
    _fields_ = [
        ("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
        ("q_stride", ctypes.c_int64 * 2), ("k_stride", ctypes.c_int64 * 2),
        ("v_stride", ctypes.c_int64 * 2),
        ("q_norm", ctypes.c_int32), ("k_norm", ctypes.c_int32),
        ("q_weight", ctypes.c_void_p), ("k_weight", ctypes.c_void_p),
        ("eps", ctypes.c_float), ("weight_offset", ctypes.c_float),
        ("rope", ctypes.c_void_p), ("positions", ctypes.c_void_p), ("pos_stride", ctypes.c_int64),
        ("q_out", ctypes.c_void_p), ("k_out", ctypes.c_void_p),
        ("k_cache", ctypes.c_void_p), ("v_cache", ctypes.c_void_p),
        ("k_mul", ctypes.c_float), ("v_mul", ctypes.c_float),
        ("num_pages", ctypes.c_int32), ("bt_stride", ctypes.c_int32),
        ("block_table", ctypes.c_void_p), ("status", ctypes.c_void_p),
    ]


# AppendArgs as one struct.pack call (null pointers are 0): a tenth of the time that setting the
# fields one by one takes.
APPEND_ARGS = struct.Struct("@3P6q2i2P2f2Pq4P2f2i2P")
assert APPEND_ARGS.size == ctypes.sizeof(AppendArgs)


_lib = None
_lock = threading.Lock()


def lib() -> ctypes.CDLL:
    """Load the CUDA library (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(
                    f"{LIB_PATH} is missing: build it with split_kv_flash_decode_gb300.build.build()"
                    " (nvcc, sm_103a); there is no fallback implementation")
            L = ctypes.CDLL(LIB_PATH)
            vp, i32, u32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_uint32, ctypes.c_size_t
            L.fd_plan.argtypes = [ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                  ctypes.POINTER(i32), ctypes.POINTER(i32), ctypes.c_int, u32,
                                  ctypes.c_int, ctypes.c_int, ctypes.POINTER(vp)]
            L.fd_plan.restype = ctypes.c_int
            L.fd_plan_destroy.argtypes = [vp]
            L.fd_plan_destroy.restype = ctypes.c_int
            L.fd_workspace_bytes.argtypes = [vp]
            L.fd_workspace_bytes.restype = sz
            L.fd_workspace_init.argtypes = [vp, vp, vp]
            L.fd_workspace_init.restype = ctypes.c_int
            L.fd_decode.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp]
            L.fd_decode.restype = ctypes.c_int
            L.fd_workspace_status.argtypes = [vp, vp, vp, ctypes.POINTER(i32)]
            L.fd_workspace_status.restype = ctypes.c_int
            L.fd_strerror.argtypes = [ctypes.c_int]
            L.fd_strerror.restype = ctypes.c_char_p
            L.fd_plan_get_info.argtypes = [vp, ctypes.POINTER(PlanInfo)]
            L.fd_plan_get_info.restype = ctypes.c_int
            L.fd_plan_get_range.argtypes = [vp, ctypes.c_int, ctypes.c_int, ctypes.POINTER(i32),
                                            ctypes.POINTER(i32)]
            L.fd_plan_get_range.restype = ctypes.c_int
            L.fd_plan_paged.argtypes = [ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                        ctypes.POINTER(i32), ctypes.POINTER(i32), ctypes.c_int,
                                        ctypes.c_int, u32, ctypes.c_int, ctypes.c_int,
                                        ctypes.POINTER(vp)]
            L.fd_plan_paged.restype = ctypes.c_int
            L.fd_decode_paged.argtypes = [vp, vp, vp, vp, ctypes.c_int, vp, ctypes.c_int, vp, vp,
                                          vp, vp]
            L.fd_decode_paged.restype = ctypes.c_int
            L.fd_decode_noalloc.argtypes = [vp, vp, vp, vp, vp, vp, vp]
            L.fd_decode_noalloc.restype = ctypes.c_int
            L.fd_noalloc_status.argtypes = [vp, vp, ctypes.POINTER(i32)]
            L.fd_noalloc_status.restype = ctypes.c_int
            L.fd_rows_plan.argtypes = [ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                       ctypes.POINTER(i32), ctypes.POINTER(i32),
                                       ctypes.POINTER(i32), ctypes.c_int, ctypes.c_int,
                                       ctypes.POINTER(vp)]
            L.fd_rows_plan.restype = ctypes.c_int
            L.fd_rows_destroy.argtypes = [vp]
            L.fd_rows_destroy.restype = ctypes.c_int
            L.fd_rows_get_info.argtypes = [vp, ctypes.POINTER(RowsInfo)]
            L.fd_rows_get_info.restype = ctypes.c_int
            L.fd_append.argtypes = [vp, vp, vp]  # byref(AppendArgs), or its bytes (APPEND_ARGS)
            L.fd_append.restype = ctypes.c_int
            L.fd_gather.argtypes = [vp, vp, vp, ctypes.c_int, vp, ctypes.c_int, vp, vp, vp, vp]
            L.fd_gather.restype = ctypes.c_int
            L.fd_tree_plan.argtypes = [ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                       ctypes.POINTER(i32), ctypes.POINTER(i32), ctypes.c_int,
                                       ctypes.c_int, ctypes.c_int, ctypes.POINTER(vp)]
            L.fd_tree_plan.restype = ctypes.c_int
            L.fd_tree_destroy.argtypes = [vp]
            L.fd_tree_destroy.restype = ctypes.c_int
            L.fd_tree_test_skip_loads.argtypes = [vp]
            L.fd_tree_test_skip_loads.restype = ctypes.c_int
            L.fd_tree_get_info.argtypes = [vp, ctypes.POINTER(TreeInfo)]
            L.fd_tree_get_info.restype = ctypes.c_int
            L.fd_tree_decode.argtypes = [vp, vp, vp, vp, ctypes.c_int, vp, ctypes.c_int, vp, vp, vp,
                                         vp, vp, vp]
            L.fd_tree_decode.restype = ctypes.c_int
            L.fd_tree_verify.argtypes = [vp, vp, ctypes.c_int64, vp, ctypes.c_int64, ctypes.c_int,
                                         vp, vp, vp, vp, vp, vp, vp]
            L.fd_tree_verify.restype = ctypes.c_int
            L.fd_tree_keep.argtypes = [vp, vp, vp, ctypes.c_int, vp, ctypes.c_int, vp, ctypes.c_int,
                                       vp, vp, vp]
            L.fd_tree_keep.restype = ctypes.c_int
            L.fd_version.argtypes = []
            L.fd_version.restype = ctypes.c_int
            _lib = L
    return _lib


def strerror(status: int) -> str:
    return lib().fd_strerror(int(status)).decode()


def _check(rc: int, where: str) -> None:
    if rc != FD_OK:
        raise FdError(rc, where)


def _i32_array(values, n: int):
    try:
        return (ctypes.c_int32 * n).from_buffer_copy(struct.pack(f"{n}i", *map(int, values)))
    except struct.error:  # ctypes would wrap what does not fit
        raise FdError(FD_ERR_INVALID, "a length outside int32") from None


def _ptr(t) -> int:
    """Device address of a tensor (or an int address, or None -> 0)."""
    if t is None:
        return 0
    if isinstance(t, int):
        return t
    return int(t.data_ptr())


def _stream(stream) -> int:
    if stream is None:
        import torch
        return int(torch.cuda.current_stream().cuda_stream)
    if isinstance(stream, int):
        return stream
    return int(stream.cuda_stream)


class Plan:
    """Owns one fd_plan_t handle (fd_plan_destroy on close / garbage collection)."""

    def __init__(self, handle: int):
        self.handle = handle
        info = PlanInfo()
        _check(lib().fd_plan_get_info(handle, ctypes.byref(info)), "fd_plan_get_info")
        self.info = {name: getattr(info, name) for name, _ in PlanInfo._fields_}
        self.info["stream"] = int(info.records_per_segment == 0)

    @property
    def workspace_bytes(self) -> int:
        return fd_workspace_bytes(self)

    def range(self, b: int, slot: int):
        return fd_plan_get_range(self, b, slot)

    def close(self) -> None:
        if self.handle:
            lib().fd_plan_destroy(self.handle)
            self.handle = 0

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def fd_plan(B, Hq, Hkv, d, seqlens, W, dtype="f16", flags=0, chunks=0, num_sms=0) -> Plan:
    """fd_plan: validate a decode shape and build its work decomposition (host only)."""
    seqlens = list(seqlens)
    W = [W] * B if isinstance(W, int) else list(W)
    if len(seqlens) != B or len(W) != B:
        raise FdError(FD_ERR_INVALID, "fd_plan: seqlens and W need B entries")
    handle = ctypes.c_void_p()
    rc = lib().fd_plan(int(B), int(Hq), int(Hkv), int(d), _i32_array(seqlens, B),
                       _i32_array(W, B), DTYPES[dtype] if isinstance(dtype, str) else int(dtype),
                       int(flags), int(chunks), int(num_sms), ctypes.byref(handle))
    _check(rc, "fd_plan")
    return Plan(handle.value)


def fd_plan_paged(B, Hq, Hkv, d, seqlens, W, page_size, dtype="f16", flags=0, chunks=0,
                  num_sms=0) -> Plan:
    """fd_plan_paged: plan a decode over a paged KV cache (host only)."""
    seqlens = list(seqlens)
    W = [W] * B if isinstance(W, int) else list(W)
    if len(seqlens) != B or len(W) != B:
        raise FdError(FD_ERR_INVALID, "fd_plan_paged: seqlens and W need B entries")
    handle = ctypes.c_void_p()
    rc = lib().fd_plan_paged(int(B), int(Hq), int(Hkv), int(d), _i32_array(seqlens, B),
                             _i32_array(W, B), int(page_size),
                             DTYPES[dtype] if isinstance(dtype, str) else int(dtype), int(flags),
                             int(chunks), int(num_sms), ctypes.byref(handle))
    _check(rc, "fd_plan_paged")
    return Plan(handle.value)


def fd_decode_paged(plan: Plan, q, k_pages, v_pages, num_pages, block_table, bt_stride, out, lse,
                    workspace, stream=None) -> None:
    """fd_decode_paged: the fused decode over a paged cache (block tables)."""
    _check(lib().fd_decode_paged(plan.handle, _ptr(q), _ptr(k_pages), _ptr(v_pages),
                                 int(num_pages), _ptr(block_table), int(bt_stride), _ptr(out),
                                 _ptr(lse), _ptr(workspace), _stream(stream)), "fd_decode_paged")


def fd_plan_destroy(plan: Plan) -> None:
    plan.close()


def fd_workspace_bytes(plan: Plan) -> int:
    return int(lib().fd_workspace_bytes(plan.handle))


def fd_workspace_init(plan: Plan, workspace, stream=None) -> None:
    _check(lib().fd_workspace_init(plan.handle, _ptr(workspace), _stream(stream)),
           "fd_workspace_init")


def fd_decode(plan: Plan, q, k, v, out, lse, workspace, stream=None) -> None:
    """fd_decode: one fused launch on `stream` (default: torch's current stream)."""
    _check(lib().fd_decode(plan.handle, _ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse),
                           _ptr(workspace), _stream(stream)), "fd_decode")


def fd_decode_noalloc(plan: Plan, q, k, v, out, lse, stream=None) -> None:
    """fd_decode_noalloc: the fused decode with the library's static device scratch
    (for callers that cannot allocate device memory; see include/fd.h)."""
    _check(lib().fd_decode_noalloc(plan.handle, _ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse),
                                   _stream(stream)), "fd_decode_noalloc")


def fd_noalloc_status(plan: Plan, stream=None) -> int:
    """fd_noalloc_status: status of the last fd_decode_noalloc call (synchronises)."""
    st = ctypes.c_int32(0)
    _check(lib().fd_noalloc_status(plan.handle, _stream(stream), ctypes.byref(st)),
           "fd_noalloc_status")
    return st.value


def fd_workspace_status(plan: Plan, workspace, stream=None) -> int:
    st = ctypes.c_int32(0)
    _check(lib().fd_workspace_status(plan.handle, _ptr(workspace), _stream(stream),
                                     ctypes.byref(st)), "fd_workspace_status")
    return st.value


def fd_plan_get_range(plan: Plan, b: int, slot: int):
    lo, hi = ctypes.c_int32(0), ctypes.c_int32(0)
    _check(lib().fd_plan_get_range(plan.handle, int(b), int(slot), ctypes.byref(lo),
                                   ctypes.byref(hi)), "fd_plan_get_range")
    return lo.value, hi.value


class Rows:
    """Owns one fd_rows_t handle (fd_rows_destroy on close / garbage collection)."""

    def __init__(self, handle: int):
        self.handle = handle
        info = RowsInfo()
        _check(lib().fd_rows_get_info(handle, ctypes.byref(info)), "fd_rows_get_info")
        self.tokens, self.cache_bytes = info.tokens, info.cache_bytes

    def close(self) -> None:
        if self.handle:
            lib().fd_rows_destroy(self.handle)
            self.handle = 0

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def fd_rows_plan(B, Hq, Hkv, d, seqlens, begin, count, page_size=0, dtype="f16") -> Rows:
    """fd_rows_plan: the rows [begin_b, begin_b + count_b) of every sequence (host only)."""
    seqlens, begin, count = list(seqlens), list(begin), list(count)
    if len(seqlens) != B or len(begin) != B or len(count) != B:
        raise FdError(FD_ERR_INVALID, "fd_rows_plan: seqlens, begin and count need B entries")
    handle = ctypes.c_void_p()
    rc = lib().fd_rows_plan(int(B), int(Hq), int(Hkv), int(d), _i32_array(seqlens, B),
                            _i32_array(begin, B), _i32_array(count, B), int(page_size),
                            DTYPES[dtype] if isinstance(dtype, str) else int(dtype),
                            ctypes.byref(handle))
    _check(rc, "fd_rows_plan")
    return Rows(handle.value)


def fd_rows_destroy(rows: Rows) -> None:
    rows.close()


def fd_rows_get_info(rows: Rows) -> dict:
    info = RowsInfo()
    _check(lib().fd_rows_get_info(rows.handle, ctypes.byref(info)), "fd_rows_get_info")
    return {"tokens": info.tokens, "cache_bytes": info.cache_bytes}


def fd_append(rows: Rows, args: AppendArgs, stream=None) -> None:
    """fd_append: norm, rotation and store of the handle's tokens (one launch)."""
    _check(lib().fd_append(rows.handle, ctypes.byref(args), _stream(stream)), "fd_append")


def fd_gather(rows: Rows, k_cache, v_cache, num_pages, block_table, bt_stride, k_out, v_out,
              status=None, stream=None) -> None:
    """fd_gather: the handle's rows of K and V back in 16 bits (one launch)."""
    _check(lib().fd_gather(rows.handle, _ptr(k_cache), _ptr(v_cache), int(num_pages),
                           _ptr(block_table), int(bt_stride), _ptr(k_out), _ptr(v_out),
                           _ptr(status), _stream(stream)), "fd_gather")


class Tree:
    """Owns one fd_tree_t handle (fd_tree_destroy on close / garbage collection)."""

    def __init__(self, handle: int):
        self.handle = handle
        self.info = fd_tree_get_info(self)

    def close(self) -> None:
        if self.handle:
            lib().fd_tree_destroy(self.handle)
            self.handle = 0

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def fd_tree_plan(B, Hq, Hkv, d, seqlens, drafts, page_size=0, dtype="f16", num_sms=0) -> Tree:
    """fd_tree_plan: the last drafts_b rows of every sequence are drafted tokens (host only)."""
    seqlens, drafts = list(seqlens), list(drafts)
    if len(seqlens) != B or len(drafts) != B:
        raise FdError(FD_ERR_INVALID, "fd_tree_plan: seqlens and drafts need B entries")
    handle = ctypes.c_void_p()
    rc = lib().fd_tree_plan(int(B), int(Hq), int(Hkv), int(d), _i32_array(seqlens, B),
                            _i32_array(drafts, B), int(page_size),
                            DTYPES[dtype] if isinstance(dtype, str) else int(dtype), int(num_sms),
                            ctypes.byref(handle))
    _check(rc, "fd_tree_plan")
    return Tree(handle.value)


def fd_tree_destroy(tree: Tree) -> None:
    tree.close()


def fd_tree_test_skip_loads(tree: Tree) -> None:
    """fd_tree_test_skip_loads: the first CTA's bounded waits run out (for tests)."""
    _check(lib().fd_tree_test_skip_loads(tree.handle), "fd_tree_test_skip_loads")


def fd_tree_get_info(tree: Tree) -> dict:
    info = TreeInfo()
    _check(lib().fd_tree_get_info(tree.handle, ctypes.byref(info)), "fd_tree_get_info")
    return {name: getattr(info, name) for name, _ in TreeInfo._fields_}


def fd_tree_decode(tree: Tree, q, k, v, num_pages, block_table, bt_stride, mask, out, lse, workspace,
                   status=None, stream=None) -> None:
    """fd_tree_decode: attention of all drafted tokens over the cache."""
    _check(lib().fd_tree_decode(tree.handle, _ptr(q), _ptr(k), _ptr(v), int(num_pages),
                                _ptr(block_table), int(bt_stride), _ptr(mask), _ptr(out), _ptr(lse),
                                _ptr(workspace), _ptr(status), _stream(stream)), "fd_tree_decode")


def fd_tree_verify(tree: Tree, target, target_stride, draft, draft_stride, vocab, tokens, parents,
                   uniform, path, emitted, count, stream=None) -> None:
    """fd_tree_verify: which drafted tokens stand, and the token that follows (one launch)."""
    _check(lib().fd_tree_verify(tree.handle, _ptr(target), int(target_stride), _ptr(draft),
                                int(draft_stride), int(vocab), _ptr(tokens), _ptr(parents),
                                _ptr(uniform), _ptr(path), _ptr(emitted), _ptr(count),
                                _stream(stream)), "fd_tree_verify")


def fd_tree_keep(tree: Tree, k_cache, v_cache, num_pages, block_table, bt_stride, path, path_stride,
                 count, status=None, stream=None) -> None:
    """fd_tree_keep: the rows of the tokens that stand move together, in place (one launch)."""
    _check(lib().fd_tree_keep(tree.handle, _ptr(k_cache), _ptr(v_cache), int(num_pages),
                              _ptr(block_table), int(bt_stride), _ptr(path), int(path_stride),
                              _ptr(count), _ptr(status), _stream(stream)), "fd_tree_keep")


def fd_version() -> int:
    return int(lib().fd_version())
