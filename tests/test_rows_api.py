"""Refusals and host logic of the cache-row calls and of 4-bit plans (no GPU: nothing launches).

Device pointers here are made-up addresses; every call returns before any CUDA call.
"""
import ctypes

import numpy as np
import pytest

import split_kv_flash_decode_gb300 as fd
from split_kv_flash_decode_gb300 import _binding as B
from split_kv_flash_decode_gb300 import build

P = 1 << 20  # a made-up, aligned address; tensors below lie 1 MiB apart


@pytest.fixture(scope="module", autouse=True)
def built_lib():
    build.build()
    return fd.lib()


def _rows(B_=2, Hq=8, Hkv=2, d=128, seqlens=(100, 40), begin=(90, 0), count=(10, 40), page=0,
          dtype="f16"):
    return fd.fd_rows_plan(B_, Hq, Hkv, d, seqlens, begin, count, page, dtype)


@pytest.mark.parametrize("change,code", [
    ({}, fd.FD_OK),
    (dict(page=16), fd.FD_OK),
    (dict(d=64, dtype="f16_e4m3kv"), fd.FD_OK),
    (dict(Hq=6), fd.FD_OK),                                        # any group
    (dict(count=(0, 0)), fd.FD_OK),
    (dict(begin=(91, 0)), fd.FD_ERR_INVALID),                      # past the end
    (dict(begin=(2 ** 31 - 1, 0)), fd.FD_ERR_INVALID),
    (dict(begin=(-1, 0)), fd.FD_ERR_INVALID),
    (dict(count=(10, -1)), fd.FD_ERR_INVALID),
    (dict(seqlens=(-100, 40)), fd.FD_ERR_INVALID),
    (dict(Hq=7), fd.FD_ERR_INVALID),
    (dict(Hkv=0), fd.FD_ERR_INVALID),
    (dict(page=-16), fd.FD_ERR_INVALID),
    (dict(dtype=3), fd.FD_ERR_INVALID),
    (dict(page=48), fd.FD_ERR_UNSUPPORTED),
    (dict(page=512), fd.FD_ERR_UNSUPPORTED),
    (dict(d=96), fd.FD_ERR_UNSUPPORTED),
    (dict(seqlens=(2 ** 31 - 1, 40)), fd.FD_ERR_UNSUPPORTED),
    (dict(B_=257, seqlens=[1] * 257, begin=[0] * 257, count=[1] * 257), fd.FD_ERR_UNSUPPORTED),
])
def test_rows_plan_validation(change, code):
    if code == fd.FD_OK:
        _rows(**change).close()
        return
    with pytest.raises(fd.FdError) as e:
        _rows(**change)
    assert e.value.status == code


def test_rows_plan_null_arguments():
    L = fd.lib()
    a = (ctypes.c_int32 * 1)(4)
    h = ctypes.c_void_p()
    assert L.fd_rows_plan(1, 8, 8, 128, None, a, a, 0, 0, ctypes.byref(h)) == fd.FD_ERR_INVALID
    assert L.fd_rows_plan(1, 8, 8, 128, a, a, a, 0, 0, None) == fd.FD_ERR_INVALID
    assert L.fd_rows_destroy(None) == fd.FD_OK
    assert L.fd_rows_get_info(None, None) == fd.FD_ERR_INVALID
    assert L.fd_append(None, None, None) == fd.FD_ERR_INVALID
    assert L.fd_gather(None, None, None, 0, None, 0, None, None, None, None) == fd.FD_ERR_INVALID


@pytest.mark.parametrize("dtype,per", [("f16", 256), ("f16_e4m3kv", 128), ("bf16_e2m1kv", 72)])
def test_rows_info_and_cache_shape(dtype, per):
    r = _rows(dtype=dtype)
    assert fd.fd_rows_get_info(r)["tokens"] == 50
    tokens = 112 + 48 if dtype.endswith("e2m1kv") else 140         # whole blocks of 16
    assert r.cache_bytes == tokens * 2 * per
    es = 2 if dtype == "f16" else 1
    assert np.prod(fd.cache_shape(dtype, 2, 128, (100, 40))) * es == r.cache_bytes
    paged = _rows(dtype=dtype, page=64)
    assert paged.cache_bytes == 64 * 2 * per
    assert np.prod(fd.cache_shape(dtype, 2, 128, None, 5, 64)) * es == 5 * paged.cache_bytes


def _args(**change):
    a = fd.AppendArgs(q=P, k=2 * P, v=3 * P, q_out=4 * P, k_out=5 * P, k_cache=6 * P, v_cache=7 * P,
                      k_mul=1.0, v_mul=1.0, eps=1e-6)
    a.q_stride[:], a.k_stride[:], a.v_stride[:] = (1024, 128), (256, 128), (256, 128)
    for name, x in change.items():
        if name.endswith("stride") and isinstance(x, tuple):
            getattr(a, name)[:] = x
        else:
            setattr(a, name, x)
    return a


def _append(rows, a):
    return fd.lib().fd_append(rows.handle, ctypes.byref(a), None)


def test_append_refusals():
    r = _rows()
    for change, code in [
        (dict(q_out=0), fd.FD_ERR_INVALID), (dict(q=0), fd.FD_ERR_INVALID),
        (dict(k=0), fd.FD_ERR_INVALID), (dict(v=0), fd.FD_ERR_INVALID),
        (dict(v_cache=0), fd.FD_ERR_INVALID), (dict(k_cache=0), fd.FD_ERR_INVALID),
        (dict(k=0, k_out=0, k_cache=0, v=0, v_cache=0, q=0, q_out=0), fd.FD_ERR_INVALID),
        (dict(k_out=0, k_cache=0, v=0, v_cache=0), fd.FD_ERR_INVALID),     # k for nothing
        (dict(q_stride=(-1024, 128)), fd.FD_ERR_INVALID),
        (dict(k_mul=2.0), fd.FD_ERR_INVALID), (dict(v_mul=0.0), fd.FD_ERR_INVALID),
        (dict(k_mul=float("nan")), fd.FD_ERR_INVALID),
        (dict(q_norm=1, eps=-1.0), fd.FD_ERR_INVALID),
        (dict(k_norm=1, weight_offset=float("inf")), fd.FD_ERR_INVALID),
        (dict(block_table=P), fd.FD_ERR_INVALID),                          # contiguous rows
        (dict(q_out=2 * P), fd.FD_ERR_INVALID),                            # overlaps k
        (dict(q_out=P + 256), fd.FD_ERR_INVALID),                          # overlaps q, shifted
        (dict(q_out=P, q_stride=(2048, 128)), fd.FD_ERR_INVALID),          # in place, not contiguous
        (dict(k_out=3 * P + 16), fd.FD_ERR_INVALID),                       # overlaps v
        (dict(k_out=4 * P + 512), fd.FD_ERR_INVALID),                      # overlaps q_out
        (dict(v_cache=6 * P + 4096), fd.FD_ERR_INVALID),                   # overlaps k_cache
        (dict(v_cache=5 * P - 16), fd.FD_ERR_INVALID),                     # overlaps k_out
        (dict(k_cache=2 * P + 256), fd.FD_ERR_INVALID),                    # overlaps k
        (dict(q=P + 8), fd.FD_ERR_ALIGN), (dict(k_cache=6 * P + 4), fd.FD_ERR_ALIGN),
        (dict(q_weight=P + 2), fd.FD_ERR_ALIGN), (dict(positions=P + 2), fd.FD_ERR_ALIGN),
        (dict(k_stride=(256, 130)), fd.FD_ERR_ALIGN), (dict(status=P + 2), fd.FD_ERR_ALIGN),
    ]:
        assert _append(r, _args(**change)) == code, change


def _rope(n=64, **change):
    freq = (ctypes.c_double * max(n, 1))(*[0.5] * n)
    axis = (ctypes.c_uint8 * max(n, 1))(*[0] * n)
    rope = fd.RopeArgs(rot_dim=2 * n, inv_freq=ctypes.addressof(freq), num_axes=1, scale=1.0)
    for name, x in change.items():
        if name == "freq0":
            freq[0] = x
        elif name == "axis0":
            axis[0] = x
            rope.axis = ctypes.addressof(axis)
        else:
            setattr(rope, name, x)
    rope.keep = (freq, axis)
    return rope


@pytest.mark.parametrize("n,change,code", [
    (64, dict(num_axes=0), fd.FD_ERR_INVALID), (64, dict(num_axes=5), fd.FD_ERR_INVALID),
    (64, dict(num_axes=2), fd.FD_ERR_INVALID),                             # needs positions
    (64, dict(scale=0.0), fd.FD_ERR_INVALID), (64, dict(scale=float("inf")), fd.FD_ERR_INVALID),
    (64, dict(inv_freq=0), fd.FD_ERR_INVALID), (64, dict(freq0=float("nan")), fd.FD_ERR_INVALID),
    (64, dict(axis0=1), fd.FD_ERR_INVALID), (64, dict(rot_dim=-16), fd.FD_ERR_INVALID),
    (72, {}, fd.FD_ERR_INVALID),                                           # rot_dim > d
    (12, {}, fd.FD_ERR_UNSUPPORTED),                                       # not a multiple of 16
])
def test_rope_refusals(n, change, code):
    rope = _rope(n, **change)
    a = _args(rope=ctypes.addressof(rope))
    assert _append(_rows(), a) == code


def test_rope_over_four_bit_cache_needs_32():
    r, rope = _rows(dtype="f16_e2m1kv"), _rope(24)
    assert _append(r, _args(rope=ctypes.addressof(rope))) == fd.FD_ERR_UNSUPPORTED
    three = _rope(64, num_axes=3)
    assert _append(r, _args(rope=ctypes.addressof(three), positions=8 * P, pos_stride=49)) == \
        fd.FD_ERR_INVALID                                                  # axes overlap


def test_paged_refusals():
    r = _rows(page=16)
    ok = dict(num_pages=9, block_table=8 * P, bt_stride=7)
    for change, code in [
        (dict(block_table=0), fd.FD_ERR_INVALID), (dict(num_pages=0), fd.FD_ERR_INVALID),
        (dict(bt_stride=6), fd.FD_ERR_INVALID), (dict(block_table=8 * P + 2), fd.FD_ERR_ALIGN),
        (dict(num_pages=2 ** 27), fd.FD_ERR_UNSUPPORTED),
    ]:
        assert _append(r, _args(**{**ok, **change})) == code, change
        t = {**ok, **change}
        assert fd.lib().fd_gather(r.handle, P, 2 * P, t["num_pages"], t["block_table"], t["bt_stride"],
                                  3 * P, 4 * P, None, None) == code, change


def test_gather_refusals():
    r = _rows()
    L = fd.lib()
    assert L.fd_gather(r.handle, None, P, 0, None, 0, P, P, None, None) == fd.FD_ERR_INVALID
    assert L.fd_gather(r.handle, P, P, 0, None, 0, P, None, None, None) == fd.FD_ERR_INVALID
    assert L.fd_gather(r.handle, P + 8, P, 0, None, 0, P, P, None, None) == fd.FD_ERR_ALIGN
    assert L.fd_gather(r.handle, P, P, 0, None, 0, P, P, P + 1, None) == fd.FD_ERR_ALIGN
    assert L.fd_gather(r.handle, P, P, 1, P, 7, P, P, None, None) == fd.FD_ERR_INVALID
    assert L.fd_gather(r.handle, P, 2 * P, 0, None, 0, 3 * P, 3 * P + 512, None, None) == fd.FD_ERR_INVALID
    assert L.fd_gather(r.handle, P, 2 * P, 0, None, 0, 3 * P, 2 * P - 512, None, None) == fd.FD_ERR_INVALID


def test_no_tokens_launch_nothing():
    r = _rows(count=(0, 0))
    assert _append(r, _args()) == fd.FD_OK
    assert fd.lib().fd_gather(r.handle, P, P, 0, None, 0, P, P, None, None) == fd.FD_OK


# ---------------------------------------------------------------------------
# 4-bit decode plans
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["f16_e2m1kv", "bf16_e2m1kv"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G", [1, 2, 4, 8, 16])
def test_four_bit_plan(dtype, d, G):
    lens, W = [5000, 0, 1, 33, 1031], [3, 1, 2, 4, 8]
    p = fd.fd_plan(5, 8 * G, 8, d, lens, W, dtype, num_sms=152)
    assert p.info["path"] == 4 and p.info["kv_bytes"] == sum(lens) * 8 * 2 * 9 * d // 16
    # By default the resident CTAs take equal runs of half tiles; W * C partials on request.
    assert p.info["stream"] == 1 and p.info["ctas"] == 152 * p.info["ctas_per_sm"]
    with pytest.raises(fd.FdError) as e:
        p.range(0, 0)
    assert e.value.status == fd.FD_ERR_UNSUPPORTED
    for flags in (fd.FD_PLAN_LITERAL_W, fd.FD_PLAN_TWO_LAUNCH, fd.FD_PLAN_WAITS, fd.FD_PLAN_NO_CLUSTER):
        assert fd.fd_plan(5, 8 * G, 8, d, lens, W, dtype, flags=flags, num_sms=152).info["stream"] == 0
    p = fd.fd_plan(5, 8 * G, 8, d, lens, W, dtype, chunks=3, num_sms=152)
    paged = fd.fd_plan_paged(5, 8 * G, 8, d, lens, W, 64, dtype, chunks=2, num_sms=152)
    for plan, unit in ((p, 16), (paged, 128)):
        assert plan.info["stream"] == 0
        C = plan.info["chunks"]
        for b, L in enumerate(lens):
            at = 0
            for slot in range(W[b] * C):
                lo, hi = plan.range(b, slot)
                assert lo == at and lo <= hi <= L and (lo % unit == 0 or lo == L)
                at = hi
            assert at == L


def test_four_bit_plan_refusals():
    def code(flags=0, d=128, G=4, dtype="f16_e2m1kv"):
        try:
            fd.fd_plan(1, 8 * G, 8, d, [100], [1], dtype, flags=flags, num_sms=152).close()
        except fd.FdError as e:
            return e.status
        return fd.FD_OK
    assert code() == fd.FD_OK and code(fd.FD_PLAN_MMA_SYNC) == fd.FD_OK
    assert code(fd.FD_PLAN_FFMA) == fd.FD_ERR_UNSUPPORTED
    assert code(fd.FD_PLAN_TCGEN05) == fd.FD_ERR_UNSUPPORTED
    assert code(d=96) == fd.FD_ERR_UNSUPPORTED and code(G=3) == fd.FD_ERR_UNSUPPORTED


def test_wrapper_refusals():
    with pytest.raises(ValueError):
        fd.Rope([1.0, 0.5], axes=[0])
    with pytest.raises(ValueError):
        fd.Rope([1.0], axes=[-1])
    with pytest.raises(ValueError):
        fd.KVRows(8, 8, 128, [4], device="cpu")
    assert B.DTYPES["f16_e2m1kv"] == fd.FD_F16_E2M1KV == 4
