"""Overlaps that fd_append and fd_gather refuse, beyond q, k, v and the caches (no GPU: made-up
addresses; every call returns before any CUDA call)."""
import ctypes

import pytest

import split_kv_flash_decode_gb300 as fd
from split_kv_flash_decode_gb300 import build

P = 1 << 20  # a made-up, aligned address; tensors below lie 1 MiB apart
LENS, BEGIN, COUNT = (100, 40), (90, 0), (10, 40)


@pytest.fixture(scope="module", autouse=True)
def built_lib():
    build.build()
    return fd.lib()


def call(page=0, **change):
    rows = fd.fd_rows_plan(2, 8, 2, 128, LENS, BEGIN, COUNT, page, "f16")
    freq = (ctypes.c_double * 64)(*[0.5] * 64)
    axis = (ctypes.c_uint8 * 64)(*[1] * 64)
    rope = fd.RopeArgs(rot_dim=128, inv_freq=ctypes.addressof(freq), axis=ctypes.addressof(axis), num_axes=2,
                       scale=1.0)
    a = fd.AppendArgs(q=P, k=2 * P, v=3 * P, q_out=4 * P, k_out=5 * P, k_cache=6 * P, v_cache=7 * P, q_norm=1,
                      k_norm=1, q_weight=8 * P, k_weight=9 * P, rope=ctypes.addressof(rope), positions=10 * P,
                      pos_stride=1000, k_mul=1.0, v_mul=1.0, eps=1e-6, status=12 * P)
    a.q_stride[:], a.k_stride[:], a.v_stride[:] = (1024, 128), (256, 128), (256, 128)
    if page:
        a.block_table, a.bt_stride, a.num_pages = 11 * P, 1000, 9
    for name, x in change.items():
        setattr(a, name, x)
    return fd.lib().fd_append(rows.handle, ctypes.byref(a), None)


@pytest.mark.parametrize("change", [
    dict(q_weight=4 * P), dict(q_weight=4 * P - 240), dict(k_weight=5 * P + 16), dict(k_weight=6 * P),
    dict(positions=4 * P + 64),
    dict(positions=5 * P - 4 * 1000),                   # the second axis begins where k_out does
    dict(positions=5 * P - 4 * (1000 + 49)),            # the last position of the second axis
    dict(status=4 * P), dict(status=7 * P + 4), dict(status=P + 8), dict(status=8 * P + 252),
    dict(status=10 * P + 4 * 1049),
], ids=str)
def test_append_refuses_outputs_over_any_input(change):
    assert call(**change) == fd.FD_ERR_INVALID


@pytest.mark.parametrize("change", [
    dict(block_table=4 * P), dict(block_table=6 * P + 64),
    dict(block_table=5 * P - 4 * 1000),                 # the second sequence's row
    dict(block_table=5 * P - 4 * 1006),                 # its last entry
    dict(status=11 * P + 4 * 1006),
], ids=str)
def test_append_refuses_outputs_over_the_page_table(change):
    assert call(page=16, **change) == fd.FD_ERR_INVALID


@pytest.mark.parametrize("table,status,k_out", [
    (3 * P, 0, 3 * P), (3 * P - 4 * 1006, 0, 3 * P), (5 * P, 3 * P + 8, 3 * P), (5 * P, 5 * P + 4, 3 * P),
    (5 * P, P, 3 * P),
])
def test_gather_refuses_outputs_over_the_page_table_and_status(table, status, k_out):
    rows = fd.fd_rows_plan(2, 8, 2, 128, LENS, BEGIN, COUNT, 16, "f16")
    assert fd.lib().fd_gather(rows.handle, P, 2 * P, 9, table, 1000, k_out, 4 * P, status, None) == \
        fd.FD_ERR_INVALID
