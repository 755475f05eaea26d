"""More of the decode over a 4-bit cache: sequences without any weight, the precision of the weights,
long sequences on both kernels, no lse.

Precision (test_weights_keep_22_bits).  For groups of up to 4 heads P.V sees every weight as the sum
of two fp16 values, off by at most 2^-22 of itself (or 2^-25, half the smallest step of the second).
Scores here are below 1/8 in the log2 domain with sum |q k| scale below 1/2, so their fp32 sums are off
by less than 8 x 2^-22 x 1/2 = 2^-20, which with ex2's 2^-22 keeps a weight within 2^-20 + 2^-22 + 2^-22
of itself; P.V's sums of at most 32 k-steps add 32 x 2^-22 max |V|.  |out - exact| is then below 2 x
1.5 x 2^-20 max |V| + 2^-17 max |V| < 2^-16 max |V|, plus the output's rounding (eps |out|; 2^-25 below the
normal values).  The values come in pairs of opposite rows, so that out, and its rounding, are small: one rounding of
the weights to 11 bits would be off by up to 2^-12 max |V|, and the test shows, in fp64 on the same
inputs, that it would not pass.
"""
import numpy as np
import pytest

import oracle
from test_kv4 import Case, f64, fd  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("sms", [0, 1])
@pytest.mark.parametrize("G,d", [(1, 64), (2, 128), (4, 128), (8, 64), (16, 128)])
def test_sequences_without_any_weight(fd, G, d, sms):  # noqa: F811
    """Every score of a sequence overflows to -inf: out is 0 and lse -inf, as for one without tokens,
    whether a CTA has the pair alone or shares it, and on the one-CTA-per-partial kernel too."""
    import torch
    c = Case(fd, "bf16_e2m1kv", d, G, 2, [3000, 100, 16, 40], [3, 1, 1, 1], seed=33, garbage=False)
    c.q = torch.full_like(c.q, 1e38)
    k = np.zeros(tuple(c.k.shape), np.uint8)
    k[:, :, :8 * d], k[:, :, 8 * d:] = 0xFF, 0x7E            # -2688 everywhere
    k[-1] = 0                                                # but in the last block of the last sequence
    c.k = torch.from_numpy(k).cuda()
    c.ref[0][:3], c.ref[1][:3] = 0, -np.inf
    c.ref[0][3] = np.repeat(c.values[1][-8:].mean(0), G, axis=0)
    c.ref[1][3] = np.log(8)
    for flags in (0, fd.FD_PLAN_TWO_LAUNCH, fd.FD_PLAN_NO_CLUSTER):
        c.check(*c.run(c.decoder(flags=flags, num_sms=sms)))


@pytest.mark.parametrize("dtype", ["f16_e2m1kv", "bf16_e2m1kv"])
@pytest.mark.parametrize("G,d", [(1, 64), (2, 128), (4, 64), (4, 128)])
def test_weights_keep_22_bits(fd, dtype, G, d):  # noqa: F811
    import torch
    lens = [2, 6, 16, 40, 200, 510]
    c = Case(fd, dtype, d, G, 2, lens, [1] * len(lens), seed=G + d)
    rs = np.random.default_rng(G)
    # Pairs of opposite values; scores of about 2^-9.
    codes, scales = oracle.quantise(rs.standard_normal((sum(lens) // 2, 2, d)))
    codes, scales = np.repeat(codes, 2, 0), np.repeat(scales, 2, 0)
    codes[1::2] ^= 8
    c.values[1] = oracle.dequantise(codes, scales)
    first = np.cumsum([0] + [-(-n // 16) * 16 for n in lens])
    row = np.concatenate([first[b] + np.arange(n) for b, n in enumerate(lens)])
    full, sfull = np.full((first[-1], 2, d), 15, np.uint8), np.full((first[-1], 2, d // 16), 0xFF, np.uint8)
    full[row], sfull[row] = codes, scales
    c.v = torch.from_numpy(oracle.pack_blocks(full, sfull, "v")).cuda()
    c.q = (c.q.float() * 2.0 ** -9).to(c.q.dtype)
    q = f64(c.q)
    ref, ref_lse = oracle.decode_reference(q, c.values[0], c.values[1], lens, "f64")
    eps = 2.0 ** -11 if dtype.startswith("f16") else 2.0 ** -8
    bound, once = np.empty_like(ref), np.empty_like(ref)
    at = 0
    for b, n in enumerate(lens):
        for h in range(c.Hq):
            k, v = c.values[0][at:at + n, h // G], c.values[1][at:at + n, h // G]
            assert (np.abs(k * q[b, h]).sum(-1) / np.sqrt(d) * np.log2(np.e)).max() < 0.5
            s = k @ q[b, h] / np.sqrt(d) * np.log2(np.e)
            assert np.abs(s).max() < 0.125
            p = np.exp2(s - s.max())
            r = p.astype(np.float16).astype(np.float64)
            once[b, h] = r @ v / r.sum()
            bound[b, h] = eps * np.abs(ref[b, h]) + 2.0 ** -25 + 2.0 ** -16 * np.abs(v).max()
        at += n
    assert (np.abs(once - ref) > 2 * bound).any(), "the test would not see weights rounded once"
    for flags in (0, fd.FD_PLAN_TWO_LAUNCH):
        out, lse = c.run(c.decoder(flags=flags))
        err = np.abs(out - ref)
        assert (err <= bound).all(), (err / bound).max()
        assert np.abs(lse - ref_lse).max() <= 1e-4


@pytest.mark.parametrize("page", [0, 64])
@pytest.mark.parametrize("dtype,G", [("f16_e2m1kv", 8), ("bf16_e2m1kv", 4)])
def test_long_sequence_on_both_kernels(fd, dtype, G, page):  # noqa: F811
    c = Case(fd, dtype, 128, G, 4, [40007, 3], [8, 1], page_size=page, seed=12)
    for chunks in (0, 5):
        dec = c.decoder(chunks=chunks)
        assert dec.info["stream"] == (chunks == 0)
        c.check(*c.run(dec))


@pytest.mark.parametrize("chunks", [0, 2])
@pytest.mark.parametrize("page", [0, 32])
def test_without_lse(fd, chunks, page):  # noqa: F811
    import torch
    c = Case(fd, "f16_e2m1kv", 128, 4, 2, [3000, 0, 77], [4, 1, 2], page_size=page, seed=14)
    dec = c.decoder(chunks=chunks)
    want, _ = c.run(dec)
    out = torch.full_like(c.q, 7.0)
    if page:
        fd.fd_decode_paged(dec.plan, c.q, c.k, c.v, c.k.shape[0], c.table, c.table.shape[1], out, None, dec.workspace)
    else:
        fd.fd_decode(dec.plan, c.q, c.k, c.v, out, None, dec.workspace)
    assert dec.status() == fd.FD_OK
    assert np.array_equal(f64(out), want)
