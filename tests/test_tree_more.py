"""More of a speculative step on the GPU: long tails of small weights, long sums, long kernels ahead, waits
that give up, the largest queries' outputs; tokens that never stand.
"""
import numpy as np
import pytest

import oracle
from test_tree import ALL, LSE_TOL, Case, f64, fd  # noqa: F401

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ attention: the weights' range

def tail_caches(dtype, L, d, rows):
    """K and V of one KV head: keys 0 but for element 0 of the given rows ({row: key}); values 1, but 0 in the
    upper half of a given row.  (k, v, the keys as stored)."""
    import torch
    if dtype.endswith("e2m1kv"):
        codes, scales = np.zeros((2, L, 1, d), np.uint8), np.full((2, L, 1, d // 16), 0x38, np.uint8)
        codes[1] = 2                                                     # 1.0
        kept = {}
        for row, key in rows.items():
            code, scale, kept[row] = (6, 0x40, 8.0) if key == 8.0 else (7, 0x3D, 9.75)
            codes[0, row, 0, 0], scales[0, row, 0, 0] = code, scale
            codes[1, row, 0, d // 2:] = 0
        return [torch.from_numpy(oracle.pack_blocks(c, s, w)).cuda() for c, s, w in zip(codes, scales, "kv")] + [kept]
    t = torch.float8_e4m3fn if dtype == "f16_e4m3kv" else torch.bfloat16 if dtype == "bf16" else torch.float16
    keys = {row: float(torch.tensor(key).to(t).float()) for row, key in rows.items()}
    k, v = torch.zeros((L, 1, d), dtype=torch.float16, device="cuda"), torch.ones((L, 1, d), dtype=torch.float16, device="cuda")
    for row, key in keys.items():
        k[row, 0, 0], v[row, 0, d // 2:] = key, 0
    if t is torch.float8_e4m3fn:
        return k.to(t).view(torch.uint8), v.to(t).view(torch.uint8), keys
    return k.to(t), v.to(t), keys


def behind_a_dominant_token(fd, dtype, L, n, G, sms, second):  # noqa: F811
    """(out, lse, weight of the tokens that lead, weight of the others for each token, score of the largest): rows 0
    and 128, the first of either softmax group's tiles, lead all others by 25 bits; `second`, row 300 leads these two by up to
    8 bits, for which the maximum in use does not move.  out's upper half is the share of the others, its lower half 1."""
    import torch
    d = 128
    rows = {0: 8.0, 128: 8.0}
    if second:
        rows[300] = 10.0 if dtype == "f16_e4m3kv" else 10.53125
    k, v, keys = tail_caches(dtype, L, d, rows)
    t16 = torch.bfloat16 if dtype.startswith("bf16") else torch.float16
    q = torch.zeros((n, G, d), dtype=t16, device="cuda")
    q[..., 0] = 24.515625
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = fd.TreeDecoder(G, 1, d, [L], [n], dtype, num_sms=sms)(q, k, v, status=status)
    assert int(status) == 0
    score = {row: float(q[0, 0, 0]) * key / np.sqrt(d) for row, key in keys.items()}
    top = max(score.values())
    assert not second or 4 < (top - score[0]) / np.log(2) < 8
    tail = (L - n + 1 + np.arange(n) - len(rows)) * np.exp(-top)         # a chain: each token sees one more
    return f64(out), f64(lse), sum(np.exp(x - top) for x in score.values()), tail, top


LONG = [(t, 131072) for t in ALL] + [("f16", 1 << 20), ("f16_e4m3kv", 1 << 20)]


@pytest.mark.parametrize("second", [False, True])
@pytest.mark.parametrize("n,G,sms", [(4, 4, 1), (33, 4, 1), (33, 4, 0)])
@pytest.mark.parametrize("dtype,L", LONG)
def test_long_tail_of_small_weights(fd, dtype, L, n, G, sms, second):  # noqa: F811
    """Each of the others weighs 2^-25 of the first, which fp16 holds only in larger units.

    A weight over these caches is off by 2^-11 of itself or, where that is more, by 2^-32 of the largest; ex2 and the
    scores' fp32 (25 bits, to 2^-22 each) by less than 2^-16 of it.  out's upper half sums equal powers of two, so
    |out - exact| <= L 2^-32 + (2^-11 + 2^-16) out and a rounding of the output."""
    out, _, lead, tail, _ = behind_a_dominant_token(fd, dtype, L, n, G, sms, second)
    eps = 2.0 ** -8 if dtype.startswith("bf16") else 2.0 ** -11
    want = (tail / (lead + tail))[:, None, None]
    err = np.abs(out[..., out.shape[2] // 2:] - want)
    assert (err <= L * 2.0 ** -32 + (2.0 ** -11 + 2.0 ** -16 + eps) * want + 2.0 ** -25).all(), (err.max(), want[0, 0, 0])


@pytest.mark.parametrize("second", [False, True])
@pytest.mark.parametrize("n,G,sms", [(4, 4, 1), (33, 4, 1), (33, 4, 0)])
@pytest.mark.parametrize("dtype,L", LONG)
def test_long_sums_of_small_addends(fd, dtype, L, n, G, sms, second):  # noqa: F811
    """The same tokens where every value is 1: the others are added to a sum that is 2^25 times each of them.  The bounds
    are test_tree.py's, for any length: sums in tensor memory go on in plain fp32 before their truncation comes to 2^-11, and
    a sum of fp32 weights of at most 64 tiles of 128, then of at most 2^13 / 64 such sums, is off by 2^-15."""
    out, lse, lead, tail, top = behind_a_dominant_token(fd, dtype, L, n, G, sms, second)
    eps = 2.0 ** -8 if dtype.startswith("bf16") else 2.0 ** -11
    err = np.abs(out[..., :out.shape[2] // 2] - 1)
    assert (err <= 2.0 ** -10 + eps).all(), err.max()
    assert np.abs(lse - (top + np.log(lead + tail))[:, None]).max() <= LSE_TOL


@pytest.mark.parametrize("n,G", [(4, 4), (33, 4)])
@pytest.mark.parametrize("dtype", ["f16", "bf16", "f16_e4m3kv"])
@pytest.mark.parametrize("page", [0, 256])
def test_long_means(fd, dtype, n, G, page):  # noqa: F811
    """2^20 tokens that weigh alike, all in one CTA: out is their mean, within the bounds of test_tree.py."""
    import torch
    d, L = 64, 1 << 20
    g = torch.Generator(device="cuda").manual_seed(5)
    v = 1 + torch.rand((L, 1, d), device="cuda", generator=g)
    t16 = torch.bfloat16 if dtype == "bf16" else torch.float16
    v = v.to(torch.float8_e4m3fn if dtype == "f16_e4m3kv" else t16)
    sums = v.double().cumsum(0)[L - n:, 0]                                # a chain: token t sees L - n + 1 + t rows
    want = (sums / (L - n + 1 + torch.arange(n, device="cuda"))[:, None]).cpu().numpy()[:, None]
    k, v = torch.zeros_like(v), v.view(torch.uint8) if dtype == "f16_e4m3kv" else v
    k, table = k.view(v.dtype), None
    if page:
        perm = torch.randperm(L // page, device="cuda", generator=g)
        k, v = (torch.empty_like(x.view(-1, page, 1, d)).index_copy_(0, perm, x.view(-1, page, 1, d)) for x in (k, v))
        table = perm.int()[None]
    q = torch.randn((n, G, d), device="cuda", generator=g).to(t16)
    out, lse = fd.TreeDecoder(G, 1, d, [L], [n], dtype, page_size=page, num_sms=1)(q, k, v, block_table=table)
    eps = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -11
    err = np.abs(f64(out) - want)
    assert (err <= 2.0 ** -10 * 2 + eps * want).all(), err.max()
    assert np.abs(f64(lse) - np.log(L - n + 1 + np.arange(n))[:, None]).max() <= LSE_TOL


@pytest.mark.parametrize("sms", [1, 2, 5])
@pytest.mark.parametrize("dtype", ALL)
def test_long_runs_of_several_items(fd, dtype, sms):  # noqa: F811
    """CTAs that go from long items to short ones and back, with one and two row tiles; lengths at which a portion's last
    tile is the one that would begin a new sum, and the one behind it."""
    if sms == 1:
        lens, drafts, page = [20000, 300, 17000, 8320, 8321, 4224, 4225], [33, 5, 4, 40, 64, 33, 64], 64
    else:
        lens, drafts, page = [33000, 1, 16640, 16641, 8448, 700, 8449], [16, 1, 8, 3, 1, 64, 20], 0
    c = Case(fd, dtype, 64 if sms == 2 else 128, 4, 2, lens, drafts, page_size=page, seed=sms)
    tree = c.tree(num_sms=sms)
    first = c.run(tree)
    c.check(*first)
    again = c.run(tree)
    assert np.array_equal(first[0], again[0]) and np.array_equal(first[1], again[1])


@pytest.mark.parametrize("dtype", ["f16", "f16_e4m3kv"])
def test_no_bounded_wait_counts_the_kernels_before(fd, dtype):  # noqa: F811
    """A call behind a kernel that lets its successors in at once and then takes over a second: waits of 1 s in the later
    kernel begin when the earlier one is done."""
    import torch
    c = Case(fd, dtype, 128, 4, 2, [700, 300], [16, 5], seed=4)
    tree = c.tree(num_sms=8)
    want = c.run(tree)
    # One CTA through one long sequence, all of its pages one page.
    q, pool = torch.randn((1, 8, 128), device="cuda").half(), torch.randn((2, 1, 256, 8, 128), device="cuda").half()
    out, lse = torch.empty_like(q), torch.empty((1, 8), device="cuda")

    def ahead(tokens):
        long = fd.TreeDecoder(8, 8, 128, [tokens], [1], "f16", page_size=256, num_sms=1)
        table = torch.zeros((1, tokens // 256), dtype=torch.int32, device="cuda")
        return lambda: long(q, *pool, block_table=table, out=out, lse=lse)
    events = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
    tokens = 1 << 18
    run = ahead(tokens)
    for e in events:
        run()
        e.record()
    torch.cuda.synchronize()
    run = ahead(min(1 << 27, int(tokens * 1500 / events[0].elapsed_time(events[1])) // 256 * 256))
    got, got_lse = torch.zeros_like(c.q), torch.zeros((21, 8), device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    events[0].record()
    run()
    tree(c.q, c.k, c.v, c.mask, out=got, lse=got_lse, status=status)
    events[1].record()
    torch.cuda.synchronize()
    assert int(status) == 0 and np.array_equal(f64(got), want[0]) and np.array_equal(f64(got_lse), want[1])
    assert events[0].elapsed_time(events[1]) > 1100


@pytest.mark.parametrize("dtype,n", [("f16", 5), ("f16", 40), ("bf16", 5), ("f16_e4m3kv", 5), ("bf16_e2m1kv", 40)])
def test_rows_of_a_wait_that_gave_up_are_nan(fd, dtype, n):  # noqa: F811
    """The first of four CTAs loads nothing (test hook): it has one of six (sequence, KV head) pairs alone and begins the
    second.  Rows of both are NaN without a look at the status word, which says so too; all others are as ever."""
    import torch
    c = Case(fd, dtype, 128, 4, 2, [3000] * 3, [n] * 3, seed=6)
    want = c.run(c.tree(num_sms=4))
    tree = c.tree(num_sms=4)
    fd.fd_tree_test_skip_loads(tree.tree)
    out, lse = torch.full((3 * n + 1, 8, 128), 7.0, dtype=c.q.dtype, device="cuda"), torch.full((3 * n + 1, 8), 7.0, device="cuda")
    status = torch.full((1,), 8, dtype=torch.int32, device="cuda")
    tree(c.q, c.k, c.v, c.mask, out=out[:-1], lse=lse[:-1], status=status)
    assert int(status) == 8 | fd.FD_TREE_TIMEOUT
    assert out[:n].isnan().all() and lse[:n].isnan().all() and (out[-1] == 7).all() and (lse[-1] == 7).all()
    assert np.array_equal(f64(out[n:-1]), want[0][n:]) and np.array_equal(f64(lse[n:-1]), want[1][n:])
    again = c.run(c.tree(num_sms=4))
    assert np.array_equal(again[0], want[0]) and np.array_equal(again[1], want[1])


def test_rows_of_a_long_run_that_gave_up_are_nan(fd):  # noqa: F811
    import torch
    c = Case(fd, "f16", 64, 2, 1, [20000], [3], seed=7)
    tree = c.tree(num_sms=1)
    fd.fd_tree_test_skip_loads(tree.tree)
    out, lse = tree(c.q, c.k, c.v, c.mask)               # no status word
    assert out.isnan().all() and lse.isnan().all()
    c.check(*c.run(c.tree(num_sms=1)))


@pytest.mark.parametrize("power", [40, 80, 118])
@pytest.mark.parametrize("dtype", ["bf16", "bf16_e2m1kv"])
def test_largest_queries_give_the_rows_that_lead(fd, dtype, power):  # noqa: F811
    """Scores whose last bit is far over 1.  A score is 64 products, each sum of them off by at most 2^-22 of their sizes
    together, and a product with the scale behind it: within 2^-16 of that sum S.  So only rows whose exact score is within
    2^-15 S of the largest (and 64, behind which a weight is 0) can have a weight, and out lies between their values;
    of a single one it is its value, rounded once.  A query of zeros gives the mean of what its token sees."""
    c = Case(fd, dtype, 64, 4, 2, [300, 40], [9, 3], seed=12, q_size=2.0 ** power)
    c.q[0, 0] = 0.0
    out, _ = c.run()
    want, _ = c.reference()
    q, (k, v), at, t, alone = f64(c.q), c.values, 0, 0, 0
    for L, n, s in zip(c.seqlens, c.drafts, c.sees):
        full = np.concatenate((np.ones((n, L - n), dtype=bool), s), 1)
        for i in range(n):
            for h in range(c.Hq):
                if not q[t + i, h].any():
                    assert (t, i, h) == (0, 0, 0)
                    v_top = np.abs(v[at:at + L, 0]).max()
                    assert (np.abs(out[0, 0] - want[0, 0]) <= 2.0 ** -10 * v_top + 2.0 ** -8 * np.abs(want[0, 0])).all()
                    continue
                sees = at + np.flatnonzero(full[i])
                terms = k[sees, h // c.G] * q[t + i, h]
                x, size = terms.sum(1) / np.sqrt(c.d), np.abs(terms).sum(1).max() / np.sqrt(c.d)
                rows = v[sees[x >= x.max() - 2.0 ** -15 * size - 64], h // c.G]
                alone += len(rows) == 1
                lo, hi = rows.min(0), rows.max(0)
                slack = 2.0 ** -8 * np.maximum(np.abs(lo), np.abs(hi)) + 2.0 ** -11 * (hi - lo)
                assert ((out[t + i, h] >= lo - slack) & (out[t + i, h] <= hi + slack)).all()
        at, t = at + L, t + n
    assert alone >= 90                                 # of the 95 rows with a query


# ------------------------------------------------------------------ verify: tokens that never stand

@pytest.mark.parametrize("u", [-0.0, -1e-30, -0.5, -2.0, -float("inf"), 5.0, float("inf"), float("nan")])
def test_tokens_without_probability_never_stand(fd, u):  # noqa: F811
    """Whatever the random number: tokens outside the vocabulary, and those that the target gives nothing."""
    import torch
    i32 = dict(dtype=torch.int32, device="cuda")
    p = torch.tensor([[0.0, 0.5, 0.5, 0.0]] * 6).cuda()
    uniform = torch.tensor([0.3] + [u] * 5).cuda()
    tree = fd.TreeDecoder(4, 2, 64, [6], [6])
    for tokens in ([1, -1, 4, 0, 3, 2 ** 31 - 1], [1, 2 ** 31 - 1, -2 ** 31, 4, -1, 3]):
        path, emitted, count = tree.verify(p, torch.tensor(tokens, **i32), uniform, parents=torch.tensor([-1, 0, 0, 0, 0, 0], **i32))
        assert int(count) == 1 and path[0].tolist() == [0] + [-1] * 5
        assert emitted[0].tolist() == [1] + [-1] * 5   # 0.3 of what the target says
    # Behind tokens that did not stand, with random numbers beyond 1: their sum goes past the whole.
    over = torch.tensor([[0.0, 0.75, 0.75, 0.0]] * 6).cuda()
    path, emitted, count = tree.verify(over, torch.tensor([1, 1, 2, 4, -1, 0], **i32), torch.tensor([0.3, 9.0, 9.0, 9.0, 9.0, 9.0]).cuda(),
                                       parents=torch.tensor([-1, 0, 0, 0, 0, 0], **i32))
    assert int(count) == 1
    # Chains with the draft's probabilities.
    draft = torch.full((6, 4), 0.25).cuda()
    for token in (-1, 4, 0, 3):
        path, emitted, count = tree.verify(p, torch.tensor([1] + [token] * 5, **i32), uniform, draft=draft)
        assert int(count) == 1 and int(emitted[0, 0]) in (1, 2)
