"""Host logic of Decoder (no GPU: what it would launch is recorded instead)."""
import contextlib

import pytest
import torch

import split_kv_flash_decode_gb300 as fd
from split_kv_flash_decode_gb300 import build
from split_kv_flash_decode_gb300 import decode as decode_mod


@pytest.fixture(scope="module", autouse=True)
def built_lib():
    build.build()
    return fd.lib()


class HostDecoder(fd.Decoder):
    """A Decoder whose tensors lie in host memory."""

    def __init__(self, seqlens, page_size=0, Hq=8, Hkv=2, d=64, dtype="f16"):
        self.device = torch.device("cpu")
        self.seqlens, self.Bsz, self.page_size = seqlens, len(seqlens), page_size
        self.Hq, self.Hkv, self.d, self.dtype = Hq, Hkv, d, dtype
        args = (self.Bsz, Hq, Hkv, d, seqlens, 1)
        self.plan = fd.fd_plan_paged(*args, page_size, dtype, num_sms=152) if page_size else \
            fd.fd_plan(*args, dtype, num_sms=152)
        self.workspace, self._home, self._others = self._zeros(), 0, {}
        self._shapes()


@pytest.fixture
def launched(monkeypatch):
    """The arguments of every call that would have been made; streams are addresses (0: the current)."""
    calls = []

    def record(index, address, call, *args):
        calls.append(args)
        return fd.FD_OK
    monkeypatch.setattr(decode_mod, "launch", record)
    monkeypatch.setattr(decode_mod, "stream_address", lambda index, stream: stream or 0)
    monkeypatch.setattr(decode_mod, "on_stream", lambda stream, device: contextlib.nullcontext())
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    return calls


@pytest.mark.parametrize("page_size", [0, 16])
def test_outputs_of_the_caller_are_checked(launched, page_size):
    """out and lse reach the kernel as addresses: only whole tensors of its types on its device do."""
    dec = HostDecoder([20, 3], page_size)
    q = torch.zeros(2, 8, 64, dtype=torch.float16)
    kv = torch.zeros((4, 16, 2, 64) if page_size else (23, 2, 64), dtype=torch.float16)
    table = torch.zeros(2, 2, dtype=torch.int32)

    def run(**kw):
        return dec.decode_paged(q, kv, kv, table, **kw) if page_size else dec(q, kv, kv, **kw)

    out, lse = torch.empty_like(q), torch.empty(2, 8)
    got = run(out=out, lse=lse)
    assert got[0] is out and got[1] is lse
    assert launched[-1][-3:] == (out.data_ptr(), lse.data_ptr(), dec.workspace.data_ptr())
    assert len(launched) == 1
    for bad in (dict(out=out[:1]), dict(out=out.bfloat16()), dict(out=out[..., :32]), dict(out=out.to("meta")),
                dict(out=torch.empty(2, 64, 8, dtype=torch.float16).transpose(1, 2)), dict(out=out.view(16, 64)),
                dict(lse=lse[:1]), dict(lse=lse.half()), dict(lse=lse.to("meta")), dict(lse=torch.empty(8, 2).T),
                dict(lse=torch.empty(2, 1).expand(2, 8)), dict(lse=lse.double())):
        with pytest.raises(ValueError):
            run(**bad)
    assert len(launched) == 1
    out, lse = run()
    assert out.shape == (2, 8, 64) and out.dtype == torch.float16 and lse.shape == (2, 8) and lse.dtype == torch.float32


def test_every_stream_has_its_own_workspace(launched, monkeypatch):
    """One workspace a stream, kept for its later calls; captured calls take what is there."""
    dec = HostDecoder([20, 3])
    q, kv = torch.zeros(2, 8, 64, dtype=torch.float16), torch.zeros(23, 2, 64, dtype=torch.float16)

    def used(stream):
        dec(q, kv, kv, stream=stream)
        return launched[-1][-1]

    first = dec.workspace.data_ptr()
    assert used(None) == first
    side, other = used(256), used(512)
    assert len({first, side, other}) == 3
    assert used(256) == side and used(512) == other and used(None) == first
    for ws in dec._others.values():
        assert ws.shape == dec.workspace.shape and not ws.any()
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
    assert used(768) == first and used(256) == side
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    assert used(768) not in (first, side, other)


def test_streams_of_other_libraries(monkeypatch):
    """Anything with a cuda_stream is a stream: its address is what counts."""
    class Stream:
        cuda_stream = 4096

    seen = []
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda address, device: seen.append(address) or "external")
    monkeypatch.setattr(torch.cuda, "stream", lambda stream: seen.append(stream) or contextlib.nullcontext())
    with decode_mod.on_stream(Stream(), torch.device("cuda", 0)):
        pass
    with decode_mod.on_stream(4096, torch.device("cuda", 0)):
        pass
    assert seen == [4096, "external"] * 2
    assert decode_mod.stream_address(0, Stream()) == 4096


def test_lengths_past_32_bits_are_refused():
    """Host lengths become int32: one that does not fit is an error, not another length."""
    for bad in ([2 ** 32 + 5], [2 ** 31], [-2 ** 32 + 1]):
        for call in (lambda: fd.fd_plan(1, 8, 8, 128, bad, 1, "f16", num_sms=152),
                     lambda: fd.fd_plan(1, 8, 8, 128, [10], bad, "f16", num_sms=152),
                     lambda: fd.fd_plan_paged(1, 8, 8, 128, bad, 1, 16, "f16", num_sms=152),
                     lambda: fd.fd_rows_plan(1, 8, 8, 128, bad, [0], [1], 0, "f16"),
                     lambda: fd.fd_rows_plan(1, 8, 8, 128, [10], bad, [1], 0, "f16"),
                     lambda: fd.fd_rows_plan(1, 8, 8, 128, [10], [0], bad, 0, "f16")):
            with pytest.raises(fd.FdError) as e:
                call()
            assert e.value.status == fd.FD_ERR_INVALID


def test_both_handles_of_the_default_stream(monkeypatch):
    """0 and 1 (the runtime's own handle) are the default stream; torch takes 1 for one of its pool."""
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda address, device: pytest.fail("external"))
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device: "default")
    monkeypatch.setattr(torch.cuda, "stream", lambda stream: contextlib.nullcontext(stream))
    for handle in (0, 1):
        with decode_mod.on_stream(handle, torch.device("cuda", 0)) as stream:
            assert stream == "default"
