"""Refusals and host logic of the speculative step's calls (no GPU: nothing launches).

Device pointers here are made-up addresses; every call returns before any CUDA call.
"""
import ctypes

import pytest

import split_kv_flash_decode_gb300 as fd
from split_kv_flash_decode_gb300 import build

P = 1 << 32  # a made-up, aligned address; tensors below lie 4 GiB apart


@pytest.fixture(scope="module", autouse=True)
def built_lib():
    build.build()
    return fd.lib()


def _tree(B_=2, Hq=8, Hkv=2, d=128, seqlens=(100, 40), drafts=(10, 40), page=0, dtype="f16", num_sms=152):
    return fd.fd_tree_plan(B_, Hq, Hkv, d, seqlens, drafts, page, dtype, num_sms)


@pytest.mark.parametrize("change,code", [
    ({}, fd.FD_OK), (dict(page=16), fd.FD_OK), (dict(d=64, dtype="f16_e4m3kv"), fd.FD_OK),
    (dict(Hq=6), fd.FD_OK), (dict(drafts=(0, 0)), fd.FD_OK), (dict(seqlens=(64, 0), drafts=(64, 0)), fd.FD_OK),
    (dict(Hq=4096, Hkv=1), fd.FD_OK),
    (dict(drafts=(10, 41)), fd.FD_ERR_INVALID), (dict(drafts=(-1, 4)), fd.FD_ERR_INVALID),
    (dict(seqlens=(-100, 40)), fd.FD_ERR_INVALID), (dict(Hq=7), fd.FD_ERR_INVALID), (dict(Hkv=0), fd.FD_ERR_INVALID),
    (dict(page=-16), fd.FD_ERR_INVALID), (dict(dtype=3), fd.FD_ERR_INVALID), (dict(num_sms=-1), fd.FD_ERR_INVALID),
    (dict(drafts=(65, 4)), fd.FD_ERR_UNSUPPORTED), (dict(page=48), fd.FD_ERR_UNSUPPORTED),
    (dict(page=512), fd.FD_ERR_UNSUPPORTED), (dict(d=96), fd.FD_ERR_UNSUPPORTED),
    (dict(Hq=4100, Hkv=1), fd.FD_ERR_UNSUPPORTED),
    (dict(seqlens=(2 ** 31 - 1, 40)), fd.FD_ERR_UNSUPPORTED),
    (dict(B_=257, seqlens=[1] * 257, drafts=[1] * 257), fd.FD_ERR_UNSUPPORTED),
], ids=str)
def test_plan_validation(change, code):
    if code == fd.FD_OK:
        _tree(**change).close()
        return
    with pytest.raises(fd.FdError) as e:
        _tree(**change)
    assert e.value.status == code


def test_null_arguments_and_info():
    L = fd.lib()
    a, h = (ctypes.c_int32 * 1)(4), ctypes.c_void_p()
    assert L.fd_tree_plan(1, 1, 1, 64, None, a, 0, 0, 152, ctypes.byref(h)) == fd.FD_ERR_INVALID
    assert L.fd_tree_plan(1, 1, 1, 64, a, None, 0, 0, 152, ctypes.byref(h)) == fd.FD_ERR_INVALID
    assert L.fd_tree_plan(1, 1, 1, 64, a, a, 0, 0, 152, None) == fd.FD_ERR_INVALID
    assert L.fd_tree_destroy(None) == fd.FD_OK
    assert L.fd_tree_get_info(None, None) == fd.FD_ERR_INVALID
    info = _tree(seqlens=(100, 40), drafts=(10, 0), dtype="bf16_e2m1kv").info
    assert info["tokens"] == 10 and info["max_drafts"] == 10 and info["kv_bytes"] == 100 * 2 * 2 * 72
    assert info["ctas"] >= 1


def _decode(tree, **change):
    a = dict(q=P, k=2 * P, v=3 * P, num_pages=0, table=0, stride=0, mask=5 * P, out=6 * P, lse=7 * P, work=8 * P, status=9 * P)
    a.update(change)
    return fd.lib().fd_tree_decode(tree.handle, a["q"], a["k"], a["v"], a["num_pages"], a["table"], a["stride"], a["mask"],
                                   a["out"], a["lse"], a["work"], a["status"], None)


Q = 2 * 50 * 8 * 128   # bytes of q and of out
KV = 2 * 140 * 2 * 128


@pytest.mark.parametrize("change,code", [
    (dict(q=0), fd.FD_ERR_INVALID), (dict(k=0), fd.FD_ERR_INVALID), (dict(v=0), fd.FD_ERR_INVALID),
    (dict(out=0), fd.FD_ERR_INVALID), (dict(table=4 * P), fd.FD_ERR_INVALID),
    (dict(q=P + 8), fd.FD_ERR_ALIGN), (dict(k=2 * P + 4), fd.FD_ERR_ALIGN), (dict(out=6 * P + 2), fd.FD_ERR_ALIGN),
    (dict(lse=7 * P + 4), fd.FD_ERR_ALIGN), (dict(work=8 * P + 8), fd.FD_ERR_ALIGN), (dict(mask=5 * P + 4), fd.FD_ERR_ALIGN),
    (dict(status=9 * P + 2), fd.FD_ERR_ALIGN),
    (dict(out=P), fd.FD_ERR_INVALID), (dict(out=P + Q - 16), fd.FD_ERR_INVALID), (dict(out=2 * P + KV - 16), fd.FD_ERR_INVALID),
    (dict(out=3 * P), fd.FD_ERR_INVALID), (dict(out=5 * P), fd.FD_ERR_INVALID), (dict(lse=6 * P + Q - 16), fd.FD_ERR_INVALID),
    (dict(lse=P), fd.FD_ERR_INVALID), (dict(status=6 * P + 4), fd.FD_ERR_INVALID), (dict(status=5 * P + 8), fd.FD_ERR_INVALID),
    (dict(status=7 * P), fd.FD_ERR_INVALID),
], ids=str)
def test_decode_refusals(change, code):
    assert _decode(_tree(), **change) == code


def test_decode_workspace_and_pages():
    assert _decode(_tree(drafts=(0, 0)), q=0, k=0, v=0, out=0) == fd.FD_OK   # nothing to do
    assert fd.lib().fd_tree_decode(None, P, P, P, 0, None, 0, None, P, None, None, None, None) == fd.FD_ERR_INVALID
    t = _tree(page=16)                                     # 7 pages for the longer sequence
    page = dict(num_pages=9, table=4 * P, stride=7)
    for change, code in [(dict(num_pages=0), fd.FD_ERR_INVALID), (dict(table=0), fd.FD_ERR_INVALID),
                         (dict(stride=6), fd.FD_ERR_INVALID), (dict(num_pages=2 ** 27), fd.FD_ERR_UNSUPPORTED),
                         (dict(table=4 * P + 2), fd.FD_ERR_ALIGN), (dict(out=4 * P), fd.FD_ERR_INVALID),
                         (dict(status=4 * P + 4 * 13), fd.FD_ERR_INVALID),
                         (dict(out=2 * P + 9 * 16 * 2 * 128 * 2 - 16), fd.FD_ERR_INVALID)]:
        assert _decode(t, **{**page, **change}) == code, change


def _verify(tree, **change):
    a = dict(target=P, ts=1000, draft=0, ds=0, vocab=1000, tokens=2 * P, parents=3 * P, uniform=4 * P, path=5 * P,
             emitted=6 * P, count=7 * P)
    a.update(change)
    return fd.lib().fd_tree_verify(tree.handle, a["target"], a["ts"], a["draft"], a["ds"], a["vocab"], a["tokens"],
                                   a["parents"], a["uniform"], a["path"], a["emitted"], a["count"], None)


@pytest.mark.parametrize("change,code", [
    (dict(target=0), fd.FD_ERR_INVALID), (dict(tokens=0), fd.FD_ERR_INVALID), (dict(uniform=0), fd.FD_ERR_INVALID),
    (dict(path=0), fd.FD_ERR_INVALID), (dict(emitted=0), fd.FD_ERR_INVALID), (dict(count=0), fd.FD_ERR_INVALID),
    (dict(vocab=0), fd.FD_ERR_INVALID), (dict(ts=999), fd.FD_ERR_INVALID), (dict(ts=-1000), fd.FD_ERR_INVALID),
    (dict(draft=8 * P, ds=1000), fd.FD_ERR_UNSUPPORTED), (dict(draft=8 * P, ds=999, parents=0), fd.FD_ERR_INVALID),
    (dict(vocab=(1 << 20) + 1, ts=1 << 21), fd.FD_ERR_UNSUPPORTED),
    (dict(target=P + 2), fd.FD_ERR_ALIGN), (dict(count=7 * P + 1), fd.FD_ERR_ALIGN),
    (dict(path=P + 4 * (49 * 1000 + 999)), fd.FD_ERR_INVALID), (dict(path=2 * P), fd.FD_ERR_INVALID),
    (dict(emitted=3 * P + 4 * 49), fd.FD_ERR_INVALID), (dict(emitted=5 * P + 4 * 79), fd.FD_ERR_INVALID),
    (dict(count=4 * P + 4), fd.FD_ERR_INVALID), (dict(count=6 * P - 4), fd.FD_ERR_INVALID),
    (dict(draft=8 * P, ds=1000, parents=0, path=8 * P + 64), fd.FD_ERR_INVALID),
], ids=str)
def test_verify_refusals(change, code):
    assert _verify(_tree(), **change) == code


def _keep(tree, **change):
    a = dict(k=P, v=2 * P, num_pages=0, table=0, stride=0, path=3 * P, ps=40, count=4 * P, status=5 * P)
    a.update(change)
    return fd.lib().fd_tree_keep(tree.handle, a["k"], a["v"], a["num_pages"], a["table"], a["stride"], a["path"], a["ps"],
                                 a["count"], a["status"], None)


@pytest.mark.parametrize("change,code", [
    (dict(k=0), fd.FD_ERR_INVALID), (dict(v=0), fd.FD_ERR_INVALID), (dict(path=0), fd.FD_ERR_INVALID),
    (dict(count=0), fd.FD_ERR_INVALID), (dict(ps=39), fd.FD_ERR_INVALID), (dict(v=P + KV - 16), fd.FD_ERR_INVALID),
    (dict(path=P + 64), fd.FD_ERR_INVALID), (dict(count=2 * P + KV - 4), fd.FD_ERR_INVALID),
    (dict(status=3 * P + 4 * 79), fd.FD_ERR_INVALID), (dict(k=P + 8), fd.FD_ERR_ALIGN), (dict(path=3 * P + 2), fd.FD_ERR_ALIGN),
    (dict(status=5 * P + 1), fd.FD_ERR_ALIGN), (dict(table=6 * P), fd.FD_ERR_INVALID),
], ids=str)
def test_keep_refusals(change, code):
    assert _keep(_tree(), **change) == code


def test_keep_without_tokens():
    assert _keep(_tree(drafts=(0, 0)), k=0, v=0) == fd.FD_OK
    assert fd.lib().fd_tree_keep(None, P, 2 * P, 0, None, 0, 3 * P, 64, 4 * P, None, None) == fd.FD_ERR_INVALID
    assert _keep(_tree(page=16), num_pages=9, table=6 * P, stride=6) == fd.FD_ERR_INVALID
