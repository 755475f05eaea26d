"""A speculative step on the GPU against the fp64 oracle: tree attention, verdicts, kept rows, and all together.

Tolerances of the attention.  Scores, softmax statistics and sums are fp32.  The weights that enter the product
with V are rounded once: fp16 2^-11 of themselves (over bf16 caches 2^-16); the sum that normalises is of the
unrounded ones.  So |out - exact| <= 2^-11 max |V| over the head's rows, plus 2^-11 max |V| for fp32 (scores
below 64 off by 128 products' 2^-24, ex2 by 2^-22: in all below 1e-5, far within), plus one rounding to the
output type (fp16 2^-11, bf16 2^-8 of the value, 2^-25 below fp16's normal values).  lse: 1e-4, as for decodes.
"""
import numpy as np
import pytest

import oracle
import workloads

pytestmark = pytest.mark.gpu

LSE_TOL = 1e-4
ALL = ["f16", "bf16", "f16_e4m3kv", "f16_e2m1kv", "bf16_e2m1kv"]


@pytest.fixture(scope="module")
def fd():
    import split_kv_flash_decode_gb300 as fd_mod
    from split_kv_flash_decode_gb300 import build
    build.build()
    return fd_mod


def f64(t):
    import torch
    return t.to(torch.float64).cpu().numpy()


def random_tree(rs, n):
    return [-1] + [int(rs.integers(max(0, i - 6), i)) for i in range(1, n)]


class Case:
    """Caches whose every row that is no token of a sequence reads as NaN, and queries of the drafted tokens."""

    def __init__(self, fd, dtype, d, G, Hkv, seqlens, drafts, page_size=0, seed=0, trees="tree", q_size=1.0):
        import torch
        rs = np.random.default_rng(seed)
        self.fd, self.dtype, self.d, self.Hq, self.Hkv, self.G = fd, dtype, d, G * Hkv, Hkv, G
        self.seqlens, self.drafts, self.page_size = list(seqlens), list(drafts), page_size
        T, N = sum(drafts), sum(seqlens)
        t16 = torch.bfloat16 if dtype.startswith("bf16") else torch.float16
        self.q = torch.from_numpy(rs.standard_normal((T, self.Hq, d)) * q_size).to(t16).cuda()
        if trees == "tree":
            self.parents = [random_tree(rs, n) for n in drafts]
            self.sees = [oracle.ancestors(p[:n]) for p, n in zip(self.parents, drafts)]
        elif trees == "chain":
            self.sees = [np.tril(np.ones((n, n), dtype=bool)) for n in drafts]
        else:  # any set of nodes, now and then none
            self.sees = [(rs.random((n, n)) < 0.4) & (rs.random((n, 1)) < 0.8) for n in drafts]
        self.mask = None
        if trees != "chain":
            bits = [sum(1 << int(j) for j in np.flatnonzero(r)) for s in self.sees for r in s]
            # Bits past the nodes of a sequence do not matter.
            past = [~((1 << n) - 1) & (2 ** 64 - 1) for n in drafts for _ in range(n)]
            bits = [x | (m if rs.random() < 0.5 else 0) for x, m in zip(bits, past)]
            self.mask = torch.tensor([x - (1 << 64) if x >> 63 else x for x in bits], dtype=torch.int64).cuda()
        self.four = dtype.endswith("e2m1kv")
        if page_size:
            need = [-(-n // page_size) for n in seqlens]
            pages = sum(need) + 3
            perm = rs.permutation(pages)
            table = np.full((len(seqlens), max(1, max(need)) + 1), -1, dtype=np.int32)
            at = 0
            for b, n in enumerate(need):
                table[b, :n] = perm[at:at + n]
                at += n
            self.table, tokens = torch.from_numpy(table).cuda(), pages * page_size
            row = [table[b, r // page_size] * page_size + r % page_size
                   for b in range(len(seqlens)) for r in range(seqlens[b])]
        else:
            self.table = None
            unit = 16 if self.four else 1
            first = np.cumsum([0] + [-(-n // unit) * unit for n in seqlens])
            tokens = max(1, int(first[-1]))
            row = [first[b] + r for b in range(len(seqlens)) for r in range(seqlens[b])]
        self.row = np.array(row, dtype=np.int64)
        self.values, caches = [], []
        for which in "kv":
            x = rs.standard_normal((N, Hkv, d)) * (rs.uniform(0.25, 1.75, d) if which == "k" else 1.0)
            if self.four:
                codes, scales = oracle.quantise(x)
                c = np.full((tokens, Hkv, d), 15, np.uint8)
                s = np.full((tokens, Hkv, d // 16), 0xFF, np.uint8)
                c[self.row], s[self.row] = codes, scales
                self.values.append(oracle.dequantise(codes, scales))
                pool, per = torch.from_numpy(oracle.pack_blocks(c, s, which)), 16
            elif dtype == "f16_e4m3kv":
                c = np.full((tokens, Hkv, d), 0x7F, np.uint8)
                c[self.row] = workloads.f32_to_e4m3_bits(x.astype(np.float32))
                self.values.append(oracle.widen(c[self.row], "e4m3"))
                pool, per = torch.from_numpy(c), 1
            else:
                y = torch.from_numpy(x).to(t16)
                self.values.append(f64(y))
                pool, per = torch.full((tokens, Hkv, d), float("nan"), dtype=t16), 1
                pool[torch.from_numpy(self.row)] = y
            if page_size:
                pool = pool.reshape(pages, page_size // per, *pool.shape[1:])
            caches.append(pool.cuda())
        self.k, self.v = caches

    def tree(self, **kw):
        return self.fd.TreeDecoder(self.Hq, self.Hkv, self.d, self.seqlens, self.drafts, self.dtype,
                                   page_size=self.page_size, **kw)

    def run(self, tree=None, **kw):
        import torch
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        out, lse = (tree or self.tree())(self.q, self.k, self.v, self.mask, block_table=self.table, status=status, **kw)
        assert int(status) == 0
        return f64(out), f64(lse)

    def reference(self):
        """By numpy products per sequence and KV head (the oracle's definition, pinned against it on the CPU)."""
        out, lse = np.zeros((sum(self.drafts), self.Hq, self.d)), np.full((sum(self.drafts), self.Hq), -np.inf)
        q, (k, v), at, t = f64(self.q), self.values, 0, 0
        for L, n, s in zip(self.seqlens, self.drafts, self.sees):
            full = np.concatenate((np.ones((n, L - n), dtype=bool), s), 1)
            for h in range(self.Hq if n else 0):
                x = q[t:t + n, h] @ k[at:at + L, h // self.G].T / np.sqrt(self.d)
                x[~full] = -np.inf
                m = x.max(1, keepdims=True)
                w = np.exp(x - np.where(np.isneginf(m), 0, m))
                z = w.sum(1, keepdims=True)
                out[t:t + n, h] = np.divide(w @ v[at:at + L, h // self.G], z, out=np.zeros((n, self.d)), where=z > 0)
                with np.errstate(divide="ignore"):
                    lse[t:t + n, h] = (m + np.log(z))[:, 0]
            at, t = at + L, t + n
        return out, lse

    def check(self, out, lse, lse_tol=LSE_TOL):
        ref, ref_lse = self.reference()
        empty = np.isneginf(ref_lse)
        assert np.array_equal(np.isneginf(lse), empty)
        assert (out[empty] == 0).all()
        top, at, t = np.zeros(out.shape[:2]), 0, 0
        for L, n in zip(self.seqlens, self.drafts):
            if n:
                top[t:t + n] = np.repeat(np.abs(self.values[1][at:at + L]).max((0, 2)), self.G)
            at, t = at + L, t + n
        eps = 2.0 ** -8 if self.dtype.startswith("bf16") else 2.0 ** -11
        err = np.abs(out - ref)
        bound = 2.0 ** -10 * top[..., None] + eps * np.abs(ref) + 2.0 ** -25
        assert (err <= bound).all(), (err - bound).max()
        assert np.abs(lse[~empty] - ref_lse[~empty]).max(initial=0.0) <= lse_tol
        # Few errors are near their bound: together they are below a rounding of the output and one of the weights.
        assert np.linalg.norm(err) <= (eps + 2.0 ** -11) * np.linalg.norm(ref)


LENS = [130, 7, 1, 64, 65, 128, 129, 255, 300, 1031, 5000, 0, 12]
DRAFTS = [5, 0, 1, 64, 64, 1, 2, 33, 64, 17, 9, 0, 12]


@pytest.mark.parametrize("G", [1, 3, 4, 16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", ALL)
def test_edge_lengths(fd, dtype, d, G):
    c = Case(fd, dtype, d, G, 2, LENS, DRAFTS, seed=G + d, trees="any" if G == 3 else "tree")
    first = c.run()
    c.check(*first)
    again = c.run()
    assert np.array_equal(first[0], again[0]) and np.array_equal(first[1], again[1])


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("dtype,d,G,Hkv", [("f16", 128, 4, 3), ("bf16", 64, 8, 1), ("f16_e4m3kv", 128, 5, 2),
                                           ("f16_e4m3kv", 64, 2, 2), ("f16_e2m1kv", 64, 4, 2),
                                           ("bf16_e2m1kv", 128, 1, 5)])
def test_paged(fd, page, dtype, d, G, Hkv):
    c = Case(fd, dtype, d, G, Hkv, LENS, DRAFTS, page_size=page, seed=page + G)
    c.check(*c.run())


@pytest.mark.parametrize("dtype", ALL)
@pytest.mark.parametrize("num_sms", [1, 2, 7, 40, 151])
def test_work_cut_anywhere(fd, dtype, num_sms):
    """Sequences shared by any number of CTAs, and CTAs with many sequences."""
    c = Case(fd, dtype, 128, 4, 2, [3000, 200, 129, 1, 40, 1100, 64, 700], [16, 40, 64, 1, 33, 7, 64, 20], seed=num_sms)
    c.check(*c.run(c.tree(num_sms=num_sms)))


@pytest.mark.parametrize("dtype", ["f16", "bf16_e2m1kv"])
def test_many_small_sequences(fd, dtype):
    """CTAs that go through many sequences of one tile and one query row."""
    for n in (1, 3):
        c = Case(fd, dtype, 64, 1, 40, [3 + 7 * b for b in range(18)], [n] * 18, seed=n)
        c.check(*c.run())
        c.check(*c.run(c.tree(num_sms=3)))


@pytest.mark.parametrize("dtype", ALL)
def test_chains_and_many_heads(fd, dtype):
    c = Case(fd, dtype, 128, 16, 3, [700, 64, 2000], [64, 64, 31], trees="chain", seed=3)
    c.check(*c.run())
    c = Case(fd, dtype, 64, 7, 1, [70, 64, 2000], [4, 1, 2], trees="chain", seed=4)
    c.check(*c.run())


@pytest.mark.parametrize("dtype", ["f16", "bf16", "bf16_e2m1kv"])
def test_query_sizes(fd, dtype):
    """Scores so large that one token takes all, and so small that all count alike."""
    for size in (30.0, 1e-4):
        c = Case(fd, dtype, 128, 4, 2, [500, 65], [20, 3], seed=8, q_size=size)
        # Scores up to 2000 are off by 2^-23 of themselves.
        c.check(*c.run(), lse_tol=1e-3 if size > 1 else LSE_TOL)


@pytest.mark.parametrize("power", [40, 80, 118])
@pytest.mark.parametrize("dtype", ["bf16", "bf16_e2m1kv"])
def test_largest_queries(fd, dtype, power):
    """Scores whose last bit is far over 1: one token takes all, with a weight of 1."""
    c = Case(fd, dtype, 64, 4, 2, [300, 40], [9, 3], seed=12, q_size=2.0 ** power)
    c.q[0, 0] = 0.0
    out, lse = c.run()
    want, want_lse = c.reference()
    assert np.isfinite(lse).all() and np.isfinite(out).all()
    # A score is a sum of 64 terms whose sizes add up to less than 2^4 times the largest of them, off by 2^-23 of that.
    assert (np.abs(lse - want_lse) <= 2.0 ** -18 * np.abs(want_lse) + LSE_TOL).all()


def test_scores_that_overflow(fd):
    """Rows whose visible scores are all -inf in fp32 weigh nothing, as rows without any."""
    import torch
    c = Case(fd, "bf16", 64, 1, 1, [200], [3], trees="chain", seed=1)
    c.q.fill_(3e38)
    c.k.fill_(-3e38)
    out, lse = c.run()
    assert np.isneginf(lse).all() and (out == 0).all()


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f16_e4m3kv", "f16_e2m1kv"])
def test_nodes_that_no_token_sees(fd, dtype):
    """Padding nodes: in no mask, their rows of K and V NaN."""
    import torch
    c = Case(fd, dtype, 128, 4, 2, [200, 64, 129], [40, 64, 64], seed=9)
    hidden = [[5, 17, 39], list(range(1, 64, 2)), [0, 63]]
    at = t = 0
    nan = {"f16_e4m3kv": 0x7F, "f16_e2m1kv": 0xFF}.get(dtype, float("nan"))
    for L, n, s, hide in zip(c.seqlens, c.drafts, c.sees, hidden):
        s[:, hide] = False
        for j in hide:
            row = int(c.row[at + L - n + j])
            for cache, which in ((c.k, "k"), (c.v, "v")):
                if c.four:
                    scale = oracle.fd_rows_oracle._offsets(which, c.d)[1][row % 16]
                    cache[row // 16, :, torch.from_numpy(np.unique(scale)).cuda()] = nan
                else:
                    cache[row] = nan
        bits = [sum(1 << int(j) for j in np.flatnonzero(r)) for r in s]
        c.mask[t:t + n] = torch.tensor([x - (1 << 64) if x >> 63 else x for x in bits]).cuda()
        at, t = at + L, t + n
    c.check(*c.run())


@pytest.mark.parametrize("dtype", ["f16", "f16_e4m3kv"])
def test_offsets_past_32_bits(fd, dtype):
    """One sequence whose last rows lie past 2^31 elements; zero keys but for two marked ones."""
    import torch
    Hkv, d, L, n = 8, 128, 2200000, 3
    assert L * Hkv * d > 2 ** 31
    kv = torch.uint8 if dtype == "f16_e4m3kv" else torch.float16
    k, v = (torch.zeros((L, Hkv, d), dtype=kv, device="cuda") for _ in "kv")
    one, eight = (0x38, 0x50) if kv == torch.uint8 else (1.0, 8.0)
    k[[5, L - 2], :, 0] = eight
    v[5], v[L - 2, :, 0] = one, one
    q = torch.zeros((n, Hkv, d), dtype=torch.float16, device="cuda")
    q[..., 0] = 128.0                                  # scores 90.5: the two tokens alone count
    out, lse = fd.TreeDecoder(Hkv, Hkv, d, [L], [n], dtype)(q, k, v)
    out = f64(out)
    assert np.abs(out[0] - 1).max() <= 2.0 ** -10      # node 0 does not see row L - 2
    assert np.abs(out[1:, :, 0] - 1).max() <= 2.0 ** -10 and np.abs(out[1:, :, 1:] - 0.5).max() <= 2.0 ** -10
    want = 8 * 128 / np.sqrt(128)
    assert np.abs(f64(lse) - (want + np.log([[1.0], [2.0], [2.0]]))).max() <= 1e-4


def test_outputs_given_and_left_alone(fd):
    import torch
    c = Case(fd, "f16", 128, 4, 2, [300, 40], [7, 5], seed=2)
    tree = c.tree()
    want = c.run(tree)
    out = torch.full((12 + 2, 8, 128), 7.0, dtype=torch.float16, device="cuda")
    lse = torch.full((12 + 2, 8), 7.0, device="cuda")
    c.run(tree, out=out[:12], lse=lse[:12])
    assert np.array_equal(f64(out[:12]), want[0]) and np.array_equal(f64(lse[:12]), want[1])
    assert (out[12:] == 7).all() and (lse[12:] == 7).all()
    # lse may be missing at the C entry.
    only = torch.empty_like(c.q)
    work = torch.empty(max(16, tree.info["workspace_bytes"]), dtype=torch.uint8, device="cuda")
    fd.fd_tree_decode(tree.tree, c.q, c.k, c.v, 0, None, 0, c.mask, only, None, work)
    assert np.array_equal(f64(only), want[0])
    empty = fd.TreeDecoder(8, 2, 128, [300, 40], [0, 0], "f16")
    got = empty(c.q[:0], c.k, c.v)
    assert got[0].shape == (0, 8, 128) and got[1].shape == (0, 8)


def test_bad_pages_read_zeros(fd):
    """Indices outside the pool fault nothing; other sequences are right."""
    import torch
    c = Case(fd, "bf16", 128, 4, 2, [300, 200], [7, 5], page_size=32, seed=2)
    want = c.run()
    c.table[0, 1], c.table[0, 2] = -5, 2 ** 31 - 1
    got = c.run()
    assert np.array_equal(got[0][7:], want[0][7:]) and np.isfinite(got[0]).all()


def test_streams_graph_and_two_calls_at_once(fd):
    import torch
    a = Case(fd, "bf16", 128, 4, 2, [3000, 40], [16, 5], seed=11)
    b = Case(fd, "f16_e2m1kv", 128, 4, 2, [2500, 90], [16, 5], page_size=64, seed=12)
    want = [a.run(), b.run()]
    trees = [a.tree(), b.tree()]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(5):
        for i, c in enumerate((a, b)):
            with torch.cuda.stream(streams[i]):
                got[i].append(trees[i](c.q, c.k, c.v, c.mask, block_table=c.table))
    for i, c in enumerate((a, b)):                      # the same plan on the other stream, given by hand
        got[i].append(trees[i](c.q, c.k, c.v, c.mask, block_table=c.table, stream=streams[1 - i]))
    torch.cuda.synchronize()
    for i in (0, 1):
        for out, lse in got[i]:
            assert np.array_equal(f64(out), want[i][0]) and np.array_equal(f64(lse), want[i][1])
    # Two graphs of one plan, replayed at once.
    graphs, outs = [], []
    for _ in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(trees[0](a.q, a.k, a.v, a.mask))
    a.q.copy_(a.q.flip(0))
    a.mask.copy_(a.mask)
    eager = [x.clone() for x in trees[0](a.q, a.k, a.v, a.mask)]
    torch.cuda.synchronize()
    for _ in range(3):
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for out, lse in outs:
        assert torch.equal(out, eager[0]) and torch.equal(lse, eager[1])


# ------------------------------------------------------------------ verify

def verdicts(fd, drafts, V, seed, tree, stride=None, kind="spiky"):
    """A call's results and the oracle's, over random rows of odd kinds."""
    import torch
    rs = np.random.default_rng(seed)
    T = sum(drafts)

    def rows():
        x = rs.standard_normal((T, V)) * (4 if kind == "spiky" else 0.1)
        e = np.exp(x - x.max(1, keepdims=True))
        e = (e / e.sum(1, keepdims=True)).astype(np.float32)
        if kind == "holes":
            e[rs.random((T, V)) < 0.7] = 0
        return e
    target = rows()
    draft = None if tree else (0.5 * target + 0.5 * rows()).astype(np.float32)
    tokens = rs.integers(0, V, T)
    parents = np.concatenate([np.array(random_tree(rs, n)[:n], dtype=np.int64) for n in drafts])
    at = 0
    for n in drafts:
        for i in range(1, n):
            up = at + (parents[at + i] if tree else i - 1)
            if draft is not None:
                draft[at + i] = (0.7 * target[up] + 0.3 * draft[at + i]).astype(np.float32)
            best = np.argsort(-target[up])[:4]
            if rs.random() < 0.8:
                tokens[at + i] = best[rs.integers(0, len(best))]
        at += n
    uniform = rs.random(T).astype(np.float32)
    uniform[rs.random(T) < 0.1] = 0
    uniform[rs.random(T) < 0.1] = np.float32(1 - 2.0 ** -24)

    def put(x):
        if stride is None:
            return torch.from_numpy(x).cuda()
        wide = torch.full((T, stride), float("nan"), device="cuda")
        wide[:, 3:3 + V] = torch.from_numpy(x)
        return wide[:, 3:3 + V]
    t = fd.TreeDecoder(4, 2, 64, [n + 5 for n in drafts], drafts)
    got = t.verify(put(target), torch.from_numpy(tokens).int().cuda(), torch.from_numpy(uniform).cuda(),
                   parents=torch.from_numpy(parents).int().cuda() if tree else None,
                   draft=None if draft is None else put(draft))
    want, at = [], 0
    for n in drafts:
        s = slice(at, at + n)
        want.append(oracle.verify_walk(target[s], tokens[s], uniform[s], list(parents[s]) if tree else None,
                                       None if draft is None else draft[s]) if n else ([], []))
        at += n
    return [x.cpu().numpy() for x in got], want


def same_verdicts(got, want):
    path, emitted, count = got
    for b, (p, e) in enumerate(want):
        assert count[b] == len(p), (b, count[b], p)
        assert list(path[b, :len(p)]) == p and (path[b, len(p):] == -1).all(), b
        assert list(emitted[b, :len(p)]) == e and (emitted[b, len(p):] == -1).all(), (b, emitted[b], e)


@pytest.mark.parametrize("tree", [True, False])
@pytest.mark.parametrize("V", [1, 2, 7, 31, 257, 2048, 2049, 50021])
def test_verify(fd, V, tree):
    for seed, kind in enumerate(["spiky", "flat", "holes"]):
        drafts = [1, 0, 64, 2, 33, 5] if V < 3000 else [1, 9, 0, 20]
        same_verdicts(*verdicts(fd, drafts, V, 10 * V + seed, tree, kind=kind))


def test_verify_without_tokens(fd):
    """Empty rows may have any strides."""
    import torch
    t = fd.TreeDecoder(4, 2, 64, [5, 0], [0, 0])
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    for p in (torch.empty((0, 7), device="cuda"), torch.empty((7, 0), device="cuda").t(), torch.empty((5, 14), device="cuda")[5:, ::2]):
        path, emitted, count = t.verify(p, none, none.float(), draft=p)
        assert path.shape == emitted.shape == (2, 0) and count.tolist() == [0, 0]


def test_verify_strides_and_many(fd):
    for tree in (True, False):
        same_verdicts(*verdicts(fd, [3, 0, 7], 501, 5, tree, stride=509))
        same_verdicts(*verdicts(fd, [1 + b % 4 for b in range(256)], 999, 6, tree))


def test_verify_largest_vocabulary(fd):
    same_verdicts(*verdicts(fd, [3, 2], 1 << 20, 7, True, kind="flat"))
    same_verdicts(*verdicts(fd, [3, 2], 1 << 20, 8, False, kind="flat"))


def by_hand(fd, target, tokens, uniform, parents=None, draft=None):
    import torch
    n = len(tokens)
    t = fd.TreeDecoder(4, 2, 64, [n], [n])
    got = t.verify(torch.tensor(target, dtype=torch.float32).cuda(), torch.tensor(tokens, dtype=torch.int32).cuda(),
                   torch.tensor(uniform, dtype=torch.float32).cuda(),
                   parents=None if parents is None else torch.tensor(parents, dtype=torch.int32).cuda(),
                   draft=None if draft is None else torch.tensor(draft, dtype=torch.float32).cuda())
    path, emitted, count = (x.cpu().numpy()[0] for x in got)
    want = oracle.verify_walk(np.array(target, dtype=np.float32), tokens, np.array(uniform, dtype=np.float32),
                              parents, None if draft is None else np.array(draft, dtype=np.float32))
    assert count == len(want[0]) and list(path[:count]) == want[0] and list(emitted[:count]) == want[1]
    return want


def test_verify_odd_rows(fd):
    nan, inf = float("nan"), float("inf")
    p = [[0.5, 0.25, 0.25, 0], [0, 0, 1, 0], [0.125, 0.125, 0.25, 0.5]]
    assert by_hand(fd, p, [9, 0, 1], [0.9, 0.5, 0.499], [-1, 0, 0]) == ([0, 2], [1, 3])
    # Tokens outside the vocabulary, parents that are none, the same token twice.
    by_hand(fd, p, [0, -1, 4], [0.9, 0.0, 0.0], [-1, 0, 0])
    by_hand(fd, p, [0, 0, 0], [0.9, 0.0, 0.0], [-1, -1, 2])
    by_hand(fd, p, [0, 0, 0], [0.9, 0.0, 0.0], [-1, 1, 7])
    by_hand(fd, [p[0]] * 5, [0, 1, 1, 1, 0], [0.6, 0.9, 0.0, 0.0, 0.99], [-1, 0, 0, 0, 0])
    # Nothing left, nothing at all; values that are no probabilities.
    by_hand(fd, [[0.75, 0], [1, 0]], [0, 0], [0.5, 0.8], [-1, 0])
    by_hand(fd, [[0.75, 0.1], [1, 0]], [0, 0], [0.5, 0.8], None, [[0, 0], [1, 0.2]])
    assert by_hand(fd, [[nan, -1.0, -inf]], [0], [0.7]) == ([0], [-1])
    by_hand(fd, [[nan, 0.5, -3.0, 0.5]], [0], [0.7])
    by_hand(fd, [[0.1, inf, 0.5, nan], [1, 0, 0, 0]], [0, 1], [0.5, 0.99], [-1, 0])
    for u in (0.0, float(np.float32(1 - 2.0 ** -24))):
        by_hand(fd, [[0.0, 0.3, 0.0, 0.7, 0.0]], [0], [u])


@pytest.mark.parametrize("draft", [False, True])
@pytest.mark.parametrize("V", [40, 5000, 131072, 1 << 20])
def test_verify_rows_that_are_no_probabilities(fd, V, draft):
    """Logits, say: sums far beyond 8.  A token of the row comes out, the same one every time."""
    import torch
    g = torch.Generator().manual_seed(V)
    target = (torch.randn((6, V), generator=g) * 4).cuda()
    tokens = torch.randint(0, V, (6,), generator=g).int().cuda()
    uniform = torch.tensor([0.999999, 0.5, 0.1, 0.99, 0.7, 0.2]).cuda()
    t = fd.TreeDecoder(4, 2, 64, [3, 2, 1], [3, 2, 1])
    kw = dict(draft=torch.ones((6, V)).cuda() * 0.5) if draft else {}
    first = [x.cpu() for x in t.verify(target, tokens, uniform, **kw)]
    path, emitted, count = first
    weights = target.clamp(0, 1).cpu()
    for b, (at, n) in enumerate([(0, 3), (3, 2), (5, 1)]):
        k = int(count[b])
        assert 1 <= k <= n and path[b, :k].tolist() == list(range(k))
        last = int(emitted[b, k - 1])
        assert 0 <= last < V and weights[at + k - 1, last] > 0
    for x, y in zip(first, t.verify(target, tokens, uniform, **kw)):
        assert torch.equal(x, y.cpu())


def test_verify_tried_tokens_leave_nothing(fd):
    """The tried tokens are all that has weight, and so little that a sum of both is not the sum of each one's units."""
    a = (2 ** 23 + 40) * 2.0 ** -63  # 0.625 units beyond a whole number of 2^-57
    for V, places in ((128, (5, 7)), (128, (5, 6)), (4000, (5, 2005)), (40, (3, 35))):
        row = [0.0] * V
        for x in places:
            row[x] = a
        for u, left in ((0.25, places[0]), (0.75, places[1])):
            assert by_hand(fd, [row] * 3, [0, *places], [u, 0.9, 0.9], [-1, 0, 0]) == ([0], [left])


def test_verify_differences_below_a_unit(fd):
    """What the target has over the draft is less than the sums' unit at every token, more at all together."""
    import torch
    V = 1 << 16
    q = torch.full((2, V), 2.0 ** -36)
    p = q + 2.0 ** -59  # an ulp
    q[:, 9] = 1.0
    t = fd.TreeDecoder(4, 2, 64, [2], [2])
    path, emitted, count = (x.cpu() for x in t.verify(p.cuda(), torch.tensor([0, 9], dtype=torch.int32).cuda(),
                                                      torch.tensor([0.5, 0.5]).cuda(), draft=q.cuda()))
    assert int(count) == 1 and path[0].tolist() == [0, -1]
    assert 0 <= int(emitted[0, 0]) < V and int(emitted[0, 0]) != 9


@pytest.mark.parametrize("u", [1.0, 5.0, -2.0, float("nan"), float("inf"), -float("inf")])
def test_verify_uniforms_out_of_range_stay_in_the_vocabulary(fd, u):
    import torch
    t = fd.TreeDecoder(4, 2, 64, [3], [3])
    p = torch.tensor([[0.0, 0.5, 0.5, 0.0]] * 3).cuda()
    path, emitted, count = t.verify(p, torch.tensor([1, 1, 2], dtype=torch.int32).cuda(), torch.full((3,), u).cuda())
    c = int(count)
    assert 1 <= c <= 3 and path[0, :c].tolist() == list(range(c))
    assert all(x in (1, 2) for x in emitted[0, :c].tolist())


# ------------------------------------------------------------------ keep

def as_rows(c, cache):
    """Every stored byte of a cache by token row: [rows, bytes]."""
    import torch
    x = cache.cpu()
    if not c.four:
        return x.reshape(-1, c.Hkv * c.d).view(torch.uint8).reshape(-1, c.Hkv * c.d * x.element_size()).numpy()
    which = "k" if cache is c.k else "v"
    codes, scales = oracle.unpack_blocks(x.reshape(-1, c.Hkv, 9 * c.d).numpy(), which)
    return np.concatenate((codes.reshape(len(codes), -1), scales.reshape(len(codes), -1)), 1)


@pytest.mark.parametrize("page", [0, 16, 64])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", ALL)
def test_keep(fd, dtype, d, page):
    import torch
    c = Case(fd, dtype, d, 2, 3, LENS, DRAFTS, page_size=page, seed=d + page)
    rs = np.random.default_rng(d + page)
    paths = [sorted(rs.choice(n, int(rs.integers(0, n + 1)), replace=False).tolist()) for n in DRAFTS]
    paths[3] = list(range(64))                         # all stand: nothing moves
    paths[4] = list(range(1, 64))                      # every row moves by one
    top = max(DRAFTS)
    path = torch.tensor([p + [77] * (top - len(p)) for p in paths], dtype=torch.int32).cuda()
    count = torch.tensor([len(p) for p in paths], dtype=torch.int32).cuda()
    before = [as_rows(c, x) for x in (c.k, c.v)]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    c.tree().keep(c.k, c.v, path, count, block_table=c.table, status=status)
    assert int(status) == 0
    for old, cache in zip(before, (c.k, c.v)):
        want, at = old.copy(), 0
        for L, n, p in zip(LENS, DRAFTS, paths):
            rows = c.row[at + L - n:at + L]
            want[rows] = oracle.keep_rows(old[rows], p)
            at += L
        assert np.array_equal(as_rows(c, cache), want)


@pytest.mark.parametrize("dtype", ["f16", "f16_e2m1kv"])
def test_keep_refuses_bad_paths_and_pages(fd, dtype):
    import torch
    c = Case(fd, dtype, 128, 2, 2, [40, 40, 40, 40, 40, 40], [6] * 6, page_size=16, seed=1)
    paths = [[0, 2, 5, 3, 4, 5], [1, 1, 2, 3, 4, 5], [-1, 2, 3, 4, 5, 6], [1, 6, 2, 3, 4, 5], [0, 2, 3, 5, 9, 9], [1, 3, 5, 0, 0, 0]]
    counts = [6, 3, 2, 2, 1000, -4]
    path = torch.tensor(paths, dtype=torch.int32).cuda()
    before = [as_rows(c, x) for x in (c.k, c.v)]
    status = torch.full((1,), 8, dtype=torch.int32, device="cuda")
    tree = c.tree()
    tree.keep(c.k, c.v, path, torch.tensor(counts, dtype=torch.int32).cuda(), block_table=c.table, status=status)
    assert int(status) == 8 | fd.FD_TREE_BAD_PATH
    for old, cache in zip(before, (c.k, c.v)):
        want = old.copy()
        for b in range(6):
            rows = c.row[40 * b + 34:40 * b + 40]
            want[rows] = oracle.keep_rows(old[rows], paths[b][:max(0, min(counts[b], 6))])
        assert np.array_equal(as_rows(c, cache), want)
    # Rows 34 .. 39 lie in the third page.
    before = [as_rows(c, x) for x in (c.k, c.v)]
    c.table[0, 2] = 10 ** 6
    path[:] = torch.tensor([1, 3, 5, 0, 0, 0], dtype=torch.int32)
    status.zero_()
    tree.keep(c.k, c.v, path, torch.tensor([3, 0, 0, 0, 0, 0], dtype=torch.int32).cuda(), block_table=c.table, status=status)
    assert int(status) == fd.FD_TREE_BAD_PAGE
    for old, cache in zip(before, (c.k, c.v)):
        assert np.array_equal(as_rows(c, cache), old)


# ------------------------------------------------------------------ a step as it is used

@pytest.mark.parametrize("dtype,page", [("f16", 0), ("bf16", 32), ("f16_e4m3kv", 64), ("bf16_e2m1kv", 16)])
def test_steps_equal_decodes_of_what_stands(fd, dtype, page):
    """Append drafts, attend, judge, keep, over several steps: each node's output is the decode of its path in a
    cache without drafts, and the cache at the end holds the tokens that stand, to the bit."""
    import torch
    G, Hkv, d, V, Hq = 4, 2, 128, 300, 8
    rs = np.random.default_rng(4)
    g = torch.Generator().manual_seed(4)
    t16 = torch.bfloat16 if dtype.startswith("bf16") else torch.float16
    rope = fd.Rope(10000.0 ** (-np.arange(64) / 64))
    prefix = [37, 0, 130]
    most = [x + 40 for x in prefix]
    table = None
    if page:
        per = -(-max(most) // page)
        table = torch.from_numpy(rs.permutation(3 * per).astype(np.int32).reshape(3, per)).cuda()
        caches = [torch.zeros(fd.cache_shape(dtype, Hkv, d, None, 3 * per, page), dtype=torch.uint8 if "kv" in dtype else t16,
                              device="cuda") for _ in "kv"]
    # Every token's projections are a function of its id: the same token gives the same row.
    table_kv = torch.randn((V, Hq + 2 * Hkv, d), generator=g).to(t16).cuda()
    words = [rs.integers(0, V, n).tolist() for n in prefix]

    def fresh(lens):
        return [torch.zeros(fd.cache_shape(dtype, Hkv, d, lens, None if not page else 3 * per, page),
                            dtype=torch.uint8 if "kv" in dtype else t16, device="cuda") for _ in "kv"]

    def put(lens, begin, count, caches, ids, positions, bt):
        rows = fd.KVRows(Hq, Hkv, d, lens, begin, count, dtype=dtype, page_size=page)
        x = table_kv[torch.tensor(ids, dtype=torch.int64).cuda()]
        return rows.append(x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], *caches, rope=rope, block_table=bt,
                           positions=torch.tensor(positions, dtype=torch.int32).cuda())
    for step in range(3):
        drafts = [int(rs.integers(1, 12)) for _ in prefix]
        trees = [random_tree(rs, n) for n in drafts]
        masks, depths = zip(*(fd.tree_masks(t) for t in trees))
        # The prefix: the tokens that stand, but for the last (each sequence's root, drawn before).
        roots = [int(rs.integers(0, V)) for _ in prefix]
        base = [len(w) for w in words]
        lens = [x + n for x, n in zip(base, drafts)]
        ids = [[roots[b]] + rs.integers(0, V, drafts[b] - 1).tolist() for b in range(3)]
        caches = fresh(lens)
        every = [w + i for w, i in zip(words, ids)]
        where = [list(range(x)) + [x + z for z in dep] for x, dep in zip(base, depths)]
        q = put(lens, [0] * 3, lens, caches, sum(every, []), sum(where, []), table)
        at = np.cumsum([0] + lens)
        q = torch.cat([q[at[b] + base[b]:at[b + 1]] for b in range(3)])
        tree = fd.TreeDecoder(Hq, Hkv, d, lens, drafts, dtype, page_size=page)
        out, lse = tree(q, *caches, torch.tensor(sum(masks, []), dtype=torch.int64).cuda(), block_table=table)
        probs = torch.softmax(8 * torch.randn((sum(drafts), V), generator=g), -1)
        flat, t0 = sum(ids, []), 0
        for b, n in enumerate(drafts):                  # make most nodes likely
            for i in range(1, n):
                probs[t0 + trees[b][i], flat[t0 + i]] += 0.6
            t0 += n
        probs = (probs / probs.sum(-1, keepdim=True)).cuda()
        parents = torch.tensor(sum(trees, []), dtype=torch.int32).cuda()
        uniform = torch.rand(sum(drafts), generator=g).cuda()
        path, emitted, count = tree.verify(probs, torch.tensor(flat, dtype=torch.int32).cuda(), uniform, parents=parents)
        # Each node against a decode of its path, in a cache without the other nodes.
        t0 = 0
        for b, n in enumerate(drafts):
            for i in range(0, n, 3):
                nodes = np.flatnonzero(oracle.ancestors(trees[b])[i])
                line = words[b] + [ids[b][j] for j in nodes]
                alone = [torch.zeros(fd.cache_shape(dtype, Hkv, d, [len(line)]), dtype=caches[0].dtype, device="cuda") for _ in "kv"]
                r = fd.KVRows(Hq, Hkv, d, [len(line)], dtype=dtype)
                x = table_kv[torch.tensor(line).cuda()]
                r.append(x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], *alone, rope=rope)
                one, one_lse = fd.Decoder(Hq, Hkv, d, [len(line)], [1], dtype)(q[t0 + i:t0 + i + 1].contiguous(), *alone)
                # Two roundings of the output, two of the weights.
                tol = 2 * (2.0 ** -8 if dtype.startswith("bf16") else 2.0 ** -11) * np.abs(f64(one)) + 2.0 ** -9 * 4
                assert (np.abs(f64(out[t0 + i]) - f64(one[0])) <= tol).all()
                assert np.abs(f64(lse[t0 + i]) - f64(one_lse[0])).max() <= 2 * LSE_TOL
            t0 += n
        tree.keep(*caches, path, count, block_table=table)
        count = count.tolist()
        for b in range(3):
            nodes = path[b, :count[b]].tolist()
            assert emitted[b, :count[b] - 1].tolist() == [ids[b][j] for j in nodes[1:]]
            words[b] = words[b] + [ids[b][j] for j in nodes]
        # What stands, read back, is what a cache of these tokens alone holds.
        now = [len(w) for w in words]
        kept = fd.KVRows(Hq, Hkv, d, lens, [0] * 3, now, dtype=dtype, page_size=page).gather(*caches, block_table=table)
        caches = fresh(now)
        put(now, [0] * 3, now, caches, sum(words, []), sum([list(range(n)) for n in now], []), table)
        want = fd.KVRows(Hq, Hkv, d, now, dtype=dtype, page_size=page).gather(*caches, block_table=table)
        assert torch.equal(kept[0], want[0]) and torch.equal(kept[1], want[1])


def test_wrapper_checks(fd):
    import torch
    c = Case(fd, "f16", 64, 2, 2, [20, 5], [4, 5], page_size=16, seed=3)
    tree = c.tree()
    good = dict(q=c.q, k_cache=c.k, v_cache=c.v, mask=c.mask, block_table=c.table)
    for change in [dict(q=c.q[:3]), dict(q=c.q.float()), dict(q=c.q.cpu()), dict(q=c.q.transpose(0, 1)), dict(k_cache=c.k[:, :8]),
                   dict(v_cache=c.v.bfloat16()), dict(block_table=None), dict(block_table=c.table.long()),
                   dict(mask=c.mask.int()), dict(mask=c.mask[:4]), dict(mask=c.mask.cpu()), dict(out=c.q.float()),
                   dict(lse=torch.zeros(9, 4).cuda().half()), dict(status=torch.zeros(1).cuda())]:
        with pytest.raises(ValueError):
            tree(**{**good, **change})
    with pytest.raises(fd.FdError):
        tree(**{**good, "block_table": c.table[:, :1].contiguous()})
    with pytest.raises(fd.FdError):
        tree(**{**good, "out": c.q})
    p = torch.rand(9, 50).cuda()
    tok, u, up = torch.zeros(9, dtype=torch.int32).cuda(), torch.rand(9).cuda(), torch.zeros(9, dtype=torch.int32).cuda()
    judge = dict(target=p, tokens=tok, uniform=u, parents=up)
    for change in [dict(target=p[:8]), dict(target=p.half()), dict(target=p.t()), dict(target=p[0]), dict(tokens=tok.long()),
                   dict(uniform=u.double()), dict(parents=up[:3]), dict(draft=p[:, :40]), dict(path=tok), dict(count=tok)]:
        with pytest.raises(ValueError):
            tree.verify(**{**judge, **change})
    with pytest.raises(fd.FdError):
        tree.verify(**judge, draft=p)
    with pytest.raises(fd.FdError):
        tree.verify(**{**judge, "target": p[:1].expand(9, 50)})
    path, emitted, count = tree.verify(**judge)
    for change in [dict(path=path[:, :3]), dict(path=path.long()), dict(count=count.cpu()), dict(block_table=None)]:
        with pytest.raises(ValueError):
            tree.keep(**{**dict(k_cache=c.k, v_cache=c.v, path=path, count=count, block_table=c.table), **change})
    with pytest.raises(fd.FdError):
        tree.keep(c.k, c.k, path, count, block_table=c.table)
    with pytest.raises(ValueError):
        fd.TreeDecoder(4, 2, 64, [5], [1], device="cpu")
    with pytest.raises(fd.FdError):
        fd.TreeDecoder(4, 2, 64, [5], [6])
    none = fd.TreeDecoder(4, 2, 64, [5, 6], [0, 0])
    path, emitted, count = none.verify(p[:0], tok[:0], u[:0])
    assert path.shape == (2, 0) and count.tolist() == [0, 0]


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f16_e4m3kv", "f16_e2m1kv", "bf16_e2m1kv"])
def test_one_drafted_token_is_a_decode(fd, dtype):
    """A chain of one over many long sequences, each CTA through several of them, against the decode of the same cache."""
    import torch
    B, L, Hq, Hkv, d = 24, 5000, 32, 8, 128
    g = torch.Generator(device="cuda").manual_seed(3)
    t16 = torch.bfloat16 if dtype.startswith("bf16") else torch.float16
    x = torch.randn((B * L, Hq + 2 * Hkv, d), device="cuda", generator=g).to(t16)
    caches = [torch.empty(fd.cache_shape(dtype, Hkv, d, [L] * B), dtype=torch.uint8 if "kv" in dtype else t16, device="cuda")
              for _ in "kv"]
    fd.KVRows(Hq, Hkv, d, [L] * B, dtype=dtype).append(None, x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], *caches)
    q = x[L - 1::L, :Hq].contiguous()
    tree = fd.TreeDecoder(Hq, Hkv, d, [L] * B, [1] * B, dtype)
    want = fd.Decoder(Hq, Hkv, d, [L] * B, [4] * B, dtype)(q, *caches)
    for _ in range(20):
        got = tree(q, *caches)
        # Two roundings of the output and two of the weights (each 2^-11 of at most max |V| < 6); lse as for decodes.
        eps = 2.0 ** -8 if dtype.startswith("bf16") else 2.0 ** -11
        assert (np.abs(f64(got[0]) - f64(want[0])) <= 2 * eps * np.abs(f64(want[0])) + 2.0 ** -9 * 6).all()
        assert np.abs(f64(got[1]) - f64(want[1])).max() <= 2 * LSE_TOL
    # Their 2-norms are nearer: rounding errors do not line up.
    assert np.linalg.norm(f64(got[0]) - f64(want[0])) <= 2 * eps * np.linalg.norm(f64(want[0]))
