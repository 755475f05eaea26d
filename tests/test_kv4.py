"""Decode over a 4-bit cache against the fp64 oracle on the values that the cache stands for.

Tolerances.  Scores and sums are fp32; the weights that P.V multiplies are fp16, each off by at
most 2^-12 of itself, and the same weights normalise the output.  So out is a convex combination
of V rows under weights off by at most 2^-11 of themselves, |out - exact| <= 2^-11 max |V - out|
<= 2^-10 max |V| over the head's rows, plus 1e-5 max |V| for fp32 (scores below 64 off by 128
products' 2^-24, ex2 by 2^-22) and one rounding to the output type.  lse: 1e-4, as for the other
caches.  bf16 queries are brought to fp16 by a power of two: their elements below 2^-14 of the
head's largest |q| lose 2^-25 of it, within the fp32 allowance.
"""
import numpy as np
import pytest

import oracle

pytestmark = pytest.mark.gpu

LSE_TOL = 1e-4


@pytest.fixture(scope="module")
def fd():
    import split_kv_flash_decode_gb300 as fd_mod
    from split_kv_flash_decode_gb300 import build
    build.build()
    return fd_mod


def f64(t):
    import torch
    return t.to(torch.float64).cpu().numpy()


class Case:
    def __init__(self, fd, dtype, d, G, Hkv, seqlens, W, page_size=0, seed=0, garbage=True):
        import torch
        rs = np.random.default_rng(seed)
        self.fd, self.dtype, self.d, self.Hq, self.Hkv = fd, dtype, d, G * Hkv, Hkv
        self.seqlens, self.W, self.page_size = seqlens, W, page_size
        t16 = torch.float16 if dtype.startswith("f16") else torch.bfloat16
        self.q = torch.from_numpy(rs.standard_normal((len(seqlens), self.Hq, d))).to(t16).cuda()
        N = sum(seqlens)
        self.values, pools = [], []
        spare = 3
        need = [-(-n // page_size) for n in seqlens] if page_size else None
        if page_size:
            pages = sum(need) + spare
            perm = rs.permutation(pages)
            table = np.full((len(seqlens), max(1, max(need)) + 1), -1, dtype=np.int32)
            at = 0
            for b, n in enumerate(need):
                table[b, :n] = perm[at:at + n]
                at += n
            self.table = torch.from_numpy(table).cuda()
            tokens = pages * page_size
            row = [table[b, r // page_size] * page_size + r % page_size
                   for b in range(len(seqlens)) for r in range(seqlens[b])]
        else:
            self.table = None
            first = np.cumsum([0] + [-(-n // 16) * 16 for n in seqlens])
            tokens = int(first[-1])
            row = [first[b] + r for b in range(len(seqlens)) for r in range(seqlens[b])]
        row = np.array(row, dtype=np.int64)
        for which in "kv":
            x = rs.standard_normal((N, Hkv, d)) * (rs.uniform(0.25, 1.75, d) if which == "k" else 1.0)
            codes, scales = oracle.quantise(x)
            # Everything that is no token reads as NaN.
            c = np.full((tokens, Hkv, d), 15, np.uint8)
            s = np.full((tokens, Hkv, d // 16), 0xFF if garbage else 0, np.uint8)
            c[row], s[row] = codes, scales
            self.values.append(oracle.dequantise(codes, scales))
            pool = oracle.pack_blocks(c, s, which)
            if page_size:
                pool = pool.reshape(pages, page_size // 16, Hkv, 9 * d)
            pools.append(torch.from_numpy(pool).cuda())
        self.k, self.v = pools
        self.ref = oracle.decode_reference(f64(self.q), self.values[0], self.values[1], seqlens, "f64")

    def decoder(self, **kw):
        return self.fd.Decoder(self.Hq, self.Hkv, self.d, self.seqlens, self.W, self.dtype,
                               page_size=self.page_size, **kw)

    def run(self, dec):
        out, lse = dec.decode_paged(self.q, self.k, self.v, self.table) if self.page_size else \
            dec(self.q, self.k, self.v)
        assert dec.status() == self.fd.FD_OK
        return f64(out), f64(lse)

    def check(self, out, lse):
        ref, ref_lse = self.ref
        empty = np.isneginf(ref_lse)
        assert np.array_equal(np.isneginf(lse), empty)
        assert (out[empty] == 0).all()
        top = np.zeros(out.shape[:2])
        at = 0
        for b, L in enumerate(self.seqlens):
            v = np.abs(self.values[1][at:at + L])
            if L:
                top[b] = np.repeat(v.max((0, 2)), self.Hq // self.Hkv)
            at += L
        eps = 2.0 ** -11 if self.dtype.startswith("f16") else 2.0 ** -8
        bound = (2.0 ** -10 + 1e-5) * top[..., None] + eps * np.abs(ref) + 2.0 ** -25
        err = np.abs(out - ref)
        assert (err <= bound).all(), (err - bound).max()
        assert np.abs(lse[~empty] - ref_lse[~empty]).max(initial=0.0) <= LSE_TOL
        # Few errors are near their bound: together they are below a rounding of the weights.
        assert np.linalg.norm(err) <= (eps + 2.0 ** -11) * np.linalg.norm(ref)


LENS = [130, 0, 1, 15, 16, 17, 127, 128, 129, 1031, 5000]


@pytest.mark.parametrize("dtype", ["f16_e2m1kv", "bf16_e2m1kv"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G", [1, 2, 4, 8, 16])
def test_edge_lengths(fd, dtype, d, G):
    c = Case(fd, dtype, d, G, 2, LENS, [3, 1, 2, 1, 4, 2, 1, 8, 2, 4, 7], seed=G + d)
    dec = c.decoder()
    assert dec.info["path"] == 4
    first = c.run(dec)
    c.check(*first)
    again = c.run(dec)
    assert np.array_equal(first[0], again[0]) and np.array_equal(first[1], again[1])


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("dtype,d,G,Hkv", [("f16_e2m1kv", 128, 4, 3), ("bf16_e2m1kv", 64, 8, 1), ("bf16_e2m1kv", 128, 1, 5)])
def test_paged(fd, page, dtype, d, G, Hkv):
    c = Case(fd, dtype, d, G, Hkv, LENS, [2] * len(LENS), page_size=page, seed=page + G)
    for chunks in (0, 2):
        c.check(*c.run(c.decoder(chunks=chunks)))


@pytest.mark.parametrize("G,d", [(4, 128), (8, 64), (16, 128), (1, 128)])
@pytest.mark.parametrize("flags", ["two_launch", "waits", "cluster", "no_cluster", "cluster_combine", "no_pdl",
                                   "literal", "combiners", "debug"])
def test_plan_variants(fd, G, d, flags):
    W = 4 if flags == "cluster_combine" else [4, 3, 2]
    c = Case(fd, "bf16_e2m1kv" if G == 8 else "f16_e2m1kv", d, G, 2, [5000, 300, 17], W, seed=G)
    flag = {"two_launch": fd.FD_PLAN_TWO_LAUNCH, "waits": fd.FD_PLAN_WAITS, "cluster": fd.FD_PLAN_CLUSTER,
            "no_cluster": fd.FD_PLAN_NO_CLUSTER, "cluster_combine": fd.FD_PLAN_CLUSTER_COMBINE,
            "no_pdl": fd.FD_PLAN_NO_PDL, "literal": fd.FD_PLAN_LITERAL_W,
            "combiners": fd.FD_PLAN_COMBINERS[4], "debug": fd.FD_PLAN_DEBUG}[flags]
    c.check(*c.run(c.decoder(flags=flag)))


@pytest.mark.parametrize("dtype", ["f16_e2m1kv", "bf16_e2m1kv"])
def test_long_sequence_many_chunks(fd, dtype):
    c = Case(fd, dtype, 128, 8, 8, [40007], [8], seed=12)
    c.check(*c.run(c.decoder()))


def test_query_sizes(fd):
    """bf16 queries far from 1 (no fp16 value has their size), zero heads, mixed sizes in a head."""
    import torch
    c = Case(fd, "bf16_e2m1kv", 128, 4, 2, [300, 40], [2, 1], seed=8)
    # Tiny keys for the huge queries, so that the scores stay ordinary.
    q = c.q.float()
    q[0, 0] *= 1e30
    q[0, 1] *= 1e-30
    q[0, 2] = 0
    q[0, 3, ::2] *= 1e-6
    q[1] *= 1e4
    q[1, 4] = 2.0 ** -133
    c.q = q.bfloat16()
    ref, ref_lse = oracle.decode_reference(f64(c.q), c.values[0], c.values[1], c.seqlens, "f64")
    out, lse = c.run(c.decoder())
    # Large scores: fp32 keeps 2^-24 of their size (the softmax sits on its largest element), so
    # compare where the runner-up is clear, and everywhere for the ordinary heads.
    for b, h in ((0, 1), (0, 2), (0, 3), (0, 4), (0, 7), (1, 4)):
        assert np.abs(out[b, h] - ref[b, h]).max() <= 2e-2 * np.abs(ref[b, h]).max()
        assert abs(lse[b, h] - ref_lse[b, h]) <= LSE_TOL
    for b, h in ((0, 0), (1, 0), (1, 1), (1, 7)):
        assert np.isfinite(lse[b, h]) and abs(lse[b, h] / ref_lse[b, h] - 1) <= 1e-5
        assert np.abs(out[b, h] - ref[b, h]).max() <= 2e-2 * np.abs(ref[b, h]).max()


def test_nan_scales_stay_in_their_heads(fd):
    c = Case(fd, "f16_e2m1kv", 128, 4, 8, [300], [2], seed=75)
    k, v = c.k.cpu().numpy(), c.v.cpu().numpy()
    k[1, 3, 8 * 128 + 1 * 8 + 2] = 0x7F          # token 17 of KV head 3: elements 32..47
    v[12, 1, 8 * 128 + 5 * 16 + 8] = 0x7F        # token 200 of KV head 1: elements 80..95
    import torch
    c.k, c.v = torch.from_numpy(k).cuda(), torch.from_numpy(v).cuda()
    for flags in (0, fd.FD_PLAN_TWO_LAUNCH):
        out, lse = c.run(c.decoder(flags=flags))
        bad = np.zeros_like(out, dtype=bool)
        bad[0, 12:16] = True
        bad[0, 4:8, 80:96] = True
        assert np.array_equal(np.isnan(out), bad)
        assert np.isnan(lse[0, 12:16]).all() and not np.isnan(lse[0, :12]).any()
        ref = c.ref[0]
        assert np.abs(out[~bad] - ref[~bad]).max() <= 5e-3


def test_pages_outside_the_pool_read_zeros(fd):
    """A page index outside the pool reads zeros: keys of score 0, values 0, and no fault."""
    c = Case(fd, "f16_e2m1kv", 128, 4, 2, [200], [1], page_size=64, seed=3)
    c.table[0, 1], c.table[0, 2] = -1, c.k.shape[0]
    for x in c.values:
        x[64:192] = 0
    c.ref = oracle.decode_reference(f64(c.q), c.values[0], c.values[1], c.seqlens, "f64")
    c.check(*c.run(c.decoder()))


def test_noalloc_and_flash_decode_match(fd):
    import torch
    c = Case(fd, "bf16_e2m1kv", 64, 4, 2, [3000, 0, 77], [4, 1, 2], seed=14)
    dec = c.decoder()
    out, lse = dec(c.q, c.k, c.v)
    out2, lse2 = torch.empty_like(out), torch.empty_like(lse)
    fd.fd_decode_noalloc(dec.plan, c.q, c.k, c.v, out2, lse2)
    assert fd.fd_noalloc_status(dec.plan) == fd.FD_OK
    assert torch.equal(out, out2) and torch.equal(lse, lse2)
    out3, lse3 = fd.flash_decode(c.q, c.k, c.v, c.seqlens, c.W)
    assert torch.equal(out, out3) and torch.equal(lse, lse3)
    with pytest.raises(ValueError):
        dec(c.q, c.k[:-1], c.v)
    with pytest.raises(ValueError):
        dec(c.q.half(), c.k, c.v)


def test_batch_of_256(fd):
    lens = [int(x) for x in np.random.default_rng(1).integers(0, 200, 256)]
    c = Case(fd, "f16_e2m1kv", 64, 2, 1, lens, [2] * 256, seed=15)
    c.check(*c.run(c.decoder()))


@pytest.mark.parametrize("stream", [True, False])
def test_pipeline_wait_timeout_is_reported(fd, stream):
    """A tile that is never loaded (test hook): the bounded wait gives up, the status says so, every
    counter returns to zero, and the next decode on the workspace is right."""
    import torch
    c = Case(fd, "f16_e2m1kv", 128, 4, 2, [20000, 300], [4, 2], seed=16)
    chunks = 0 if stream else 1
    dec = c.decoder(flags=fd.FD_PLAN_TEST_SKIP_TILE, chunks=chunks, num_sms=8)
    assert dec.info["stream"] == stream
    out, lse = dec(c.q, c.k, c.v)
    assert dec.status() == fd.FD_ERR_TIMEOUT
    assert not dec.workspace[256:256 + 4 * 2 * 2].any()
    assert torch.isfinite(out).all() and torch.isfinite(lse).all()
    clean = fd.fd_plan(2, 8, 2, 128, c.seqlens, c.W, c.dtype, chunks=chunks, num_sms=8)
    out, lse = torch.empty_like(c.q), torch.empty((2, 8), dtype=torch.float32, device="cuda")
    fd.fd_decode(clean, c.q, c.k, c.v, out, lse, dec.workspace)
    assert fd.fd_workspace_status(clean, dec.workspace) == fd.FD_OK
    c.check(f64(out), f64(lse))


def test_stream_runs_cut_anywhere(fd):
    """Runs of half tiles that start and end inside pairs, cover whole pairs, or hold one half tile;
    empty sequences between them.  The counters are at rest after each decode."""
    for i, (lens, Hkv, sms) in enumerate([
            ([3000, 0, 0, 5, 700], 3, 7), ([0, 0, 64, 65, 63, 0], 2, 2), ([0], 4, 152), ([10000], 1, 152),
            ([1] * 100 + [4000], 1, 5), ([200, 9000], 5, 1), ([0, 0, 0], 1, 152)]):
        for G, dtype in ((2, "f16_e2m1kv"), (8, "bf16_e2m1kv"), (16, "f16_e2m1kv")):
            c = Case(fd, dtype, 64 if G == 2 else 128, G, Hkv, lens, [1] * len(lens), seed=i)
            dec = c.decoder(num_sms=sms)
            assert dec.info["stream"] == 1
            first = c.run(dec)
            c.check(*first)
            again = c.run(dec)
            assert np.array_equal(first[0], again[0]) and np.array_equal(first[1], again[1])
            assert not dec.workspace[256:256 + 4 * len(lens) * Hkv].any()


@pytest.mark.parametrize("G,d", [(1, 128), (4, 64), (8, 128), (16, 64)])
def test_scores_that_overflow_have_no_weight(fd, G, d):
    """Scores of -1e45 (-inf in fp32) in whole warps' and whole CTAs' shares of a sequence: the tokens
    with zero keys take all the weight, equal parts of it."""
    import torch
    c = Case(fd, "bf16_e2m1kv", d, G, 2, [3000, 100], [3, 1], seed=31, garbage=False)
    c.q = torch.full_like(c.q, 1e38)
    low = np.ones(188 + 7, bool)              # blocks of 16 tokens: -2688 everywhere, but zeros in some
    low[[100, 101, 150, 188 + 5]] = False
    k = np.zeros(tuple(c.k.shape), np.uint8)
    k[low, :, :8 * d], k[low, :, 8 * d:] = 0xFF, 0x7E
    c.k = torch.from_numpy(k).cuda()
    for b, (at, blocks) in enumerate([(0, [100, 101, 150]), (3000, [5])]):
        tokens = np.concatenate([at + 16 * j + np.arange(16) for j in blocks])
        mean = np.repeat(c.values[1][tokens].mean(0), G, axis=0)
        c.ref[0][b], c.ref[1][b] = mean, np.log(len(tokens))
    for flags in (0, fd.FD_PLAN_TWO_LAUNCH, fd.FD_PLAN_WAITS):
        c.check(*c.run(c.decoder(flags=flags)))


def test_outputs_come_from_the_pool_of_their_stream(fd):
    """Memory freed on the current stream may still be read there: a call on another stream does not
    take it for its outputs."""
    import torch
    c = Case(fd, "f16_e2m1kv", 128, 4, 2, [300], [2], seed=32)
    dec = c.decoder()
    side = torch.cuda.Stream()
    want = c.run(dec)
    for stream in (side, side.cuda_stream):
        freed = [torch.empty_like(c.q) for _ in range(4)] + [torch.empty(1, 8, device="cuda") for _ in range(4)]
        places = {x.data_ptr() for x in freed}
        del freed
        side.wait_stream(torch.cuda.current_stream())
        out, lse = dec(c.q, c.k, c.v, stream=stream)
        side.synchronize()
        assert not {out.data_ptr(), lse.data_ptr()} & places
        assert np.array_equal(f64(out), want[0]) and np.array_equal(f64(lse), want[1])
    out, lse = dec(c.q, c.k, c.v, stream=0)
    torch.cuda.synchronize()
    assert np.array_equal(f64(out), want[0]) and np.array_equal(f64(lse), want[1])
