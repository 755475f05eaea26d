"""Decoders on streams other than the one they were made on."""
import numpy as np
import pytest

import oracle

pytestmark = pytest.mark.gpu

BUSY = 20_000_000  # clock cycles (about 10 ms) for which a test keeps a stream at work


@pytest.fixture(scope="module")
def fd():
    import split_kv_flash_decode_gb300 as fd_mod
    from split_kv_flash_decode_gb300 import build
    build.build()
    return fd_mod


def f64(t):
    import torch
    return t.to(torch.float64).cpu().numpy()


class Inputs:
    """f16 inputs of a batch that several CTAs share, and its oracle answer."""

    def __init__(self, seed):
        import torch
        g = torch.Generator().manual_seed(seed)
        self.lens, self.W = [3000, 700], [4, 2]
        self.q = torch.randn((2, 8, 128), generator=g).half().cuda()
        self.k, self.v = (torch.randn((3700, 2, 128), generator=g).half().cuda() for _ in "kv")
        self.ref, self.ref_lse = oracle.decode_reference(f64(self.q), f64(self.k), f64(self.v), self.lens, "f64")

    def decoder(self, fd):
        return fd.Decoder(8, 2, 128, self.lens, self.W)

    def check(self, out, lse):
        assert np.abs(f64(out) - self.ref).max() <= 2e-3 and np.abs(f64(lse) - self.ref_lse).max() <= 1e-4


def test_first_call_on_another_stream(fd):
    """A new Decoder whose stream is still busy (its workspace's memory full of ones, its zeroing not
    yet run): a call on a side stream does not wait for it, and is right."""
    import torch
    x = Inputs(1)
    size = x.decoder(fd).plan.workspace_bytes
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (side, side.cuda_stream):
        junk = [torch.full((size,), 255, dtype=torch.uint8, device="cuda") for _ in range(4)]
        del junk
        torch.cuda.synchronize()
        torch.cuda._sleep(BUSY)
        dec = x.decoder(fd)
        x.check(*dec(x.q, x.k, x.v, stream=stream))
        assert dec.status() == fd.FD_OK


def test_decoder_dropped_while_a_side_stream_uses_it(fd):
    """The memory that a call in flight on a side stream works in is not handed out again."""
    import torch
    x = Inputs(2)
    side = torch.cuda.Stream()
    dec = x.decoder(fd)
    size = dec.plan.workspace_bytes
    x.check(*dec(x.q, x.k, x.v))
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(BUSY)
    out, lse = dec(x.q, x.k, x.v, stream=side)
    used = dec._workspace(side.cuda_stream).data_ptr()
    del dec
    later = [torch.full((size,), 255, dtype=torch.uint8, device="cuda") for _ in range(4)]
    assert used not in [t.data_ptr() for t in later]
    side.synchronize()
    x.check(out, lse)


def test_two_streams_at_once(fd):
    """Calls of one Decoder on two streams at the same time."""
    import torch
    x, y = Inputs(3), Inputs(4)
    dec = x.decoder(fd)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = []
    for _ in range(20):
        for z, s in zip((x, y), streams):
            with torch.cuda.stream(s):
                got.append((z, dec(z.q, z.k, z.v)))
    torch.cuda.synchronize()
    assert dec.status() == fd.FD_OK
    for z, (out, lse) in got:
        z.check(out, lse)


def test_captured_call_of_a_new_decoder(fd):
    """A graph whose only call is the Decoder's first: it allocates no workspace, and replays are right."""
    import torch
    x = Inputs(5)
    dec = x.decoder(fd)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = dec(x.q, x.k, x.v)
    assert not dec._others
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        x.check(out, lse)
    x.check(*dec(x.q, x.k, x.v))
    assert dec.status() == fd.FD_OK
