"""fd_append and fd_gather on the GPU against the fp64 oracle.

Tolerances.  One rounding to the stored type is off by at most half a step: eps / 2 |y| for
16 bits, 2^-4 |y| for E4M3, half the distance to the next code for E2M1; below the smallest
normal value, half the smallest step.  The fp32 arithmetic before it: the mean square of up to
128 elements (a chain of 8 fma and 4 or fewer sums in tree order, 13 roundings of 2^-24, halved
by the root), rsqrt (2 ulp: 2^-22), three products, and a rotation whose cos and sin are off by
4e-7 (angle kept to 2^-25 half turns, sincospif to 2 ulp) sum to below 2^-19 of |a| + |b|, the
two elements of the pair (of |y| alone where nothing rotates).
"""
import numpy as np
import pytest

import oracle
from oracle import fd_rows_oracle as ro

pytestmark = pytest.mark.gpu

FP32 = 2.0 ** -19
STEP = {"f16": (2.0 ** -11, 2.0 ** -25), "bf16": (2.0 ** -8, 2.0 ** -134), "e4m3": (2.0 ** -4, 2.0 ** -10)}


@pytest.fixture(scope="module")
def fd():
    import split_kv_flash_decode_gb300 as fd_mod
    from split_kv_flash_decode_gb300 import build
    build.build()
    return fd_mod


def q_name(dtype):
    return dtype.split("_")[0]


def q_type(dtype):
    import torch
    return torch.float16 if q_name(dtype) == "f16" else torch.bfloat16


def f64(t):
    import torch
    return t.to(torch.float64).cpu().numpy()


class Setup:
    """Inputs of one append, its caches (filled with a pattern) and where its rows lie."""

    def __init__(self, fd, dtype, d, Hq, Hkv, seqlens, begin, count, page_size=0, seed=0, spare=2):
        import torch
        g = torch.Generator().manual_seed(seed)
        self.fd, self.dtype, self.d, self.Hq, self.Hkv = fd, dtype, d, Hq, Hkv
        self.seqlens, self.begin, self.count, self.page_size = seqlens, begin, count, page_size
        T = sum(count)
        t16 = q_type(dtype)
        x = torch.randn((T, Hq + 2 * Hkv, d), generator=g).to(t16).cuda()
        self.q, self.k, self.v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
        self.weights = [(1 + 0.3 * torch.randn(d, generator=g)).to(t16).cuda() for _ in range(2)]
        self.four = dtype.endswith("e2m1kv")
        unit = 16 if self.four else 1
        if page_size:
            need = [-(-n // page_size) for n in seqlens]
            pages = sum(need) + spare
            perm = torch.randperm(pages, generator=g).tolist()
            table = torch.full((len(seqlens), max(1, max(need)) + 1), -7, dtype=torch.int32)
            for b, n in enumerate(need):
                table[b, :n] = torch.tensor(perm[:n], dtype=torch.int32)
                perm = perm[n:]
            self.table = table.cuda()
            shape = fd.cache_shape(dtype, Hkv, d, None, pages, page_size)
            place = lambda b, r: int(table[b, r // page_size]) * page_size + r % page_size  # noqa: E731
        else:
            self.table = None
            shape = fd.cache_shape(dtype, Hkv, d, seqlens)
            first = np.cumsum([0] + [-(-n // unit) * unit for n in seqlens])
            place = lambda b, r: int(first[b]) + r  # noqa: E731
        self.place = lambda begin, count: np.array(  # noqa: E731
            [place(b, r) for b in range(len(seqlens)) for r in range(begin[b], begin[b] + count[b])], dtype=np.int64)
        self.row = self.place(begin, count)
        self.pos = np.array(sum([list(range(a, a + n)) for a, n in zip(begin, count)], []), dtype=np.int64)
        fill = lambda: torch.randint(0, 256, (int(np.prod(shape)) * (1 if "kv" in dtype else 2),),  # noqa: E731
                                     dtype=torch.uint8, generator=g)
        self.bytes = [fill(), fill()]
        kv = torch.uint8 if "kv" in dtype else t16
        self.k_cache, self.v_cache = (x.clone().cuda().view(kv).view(shape) for x in self.bytes)
        self.rows = fd.KVRows(Hq, Hkv, d, seqlens, begin, count, dtype, page_size)

    def append(self, **kw):
        return self.rows.append(self.q, self.k, self.v, self.k_cache, self.v_cache,
                                block_table=self.table, **kw)

    def stored(self):
        """Values [T, Hkv, d] of the call's rows in both caches, with (codes, scales) for 4 bits; every
        other byte of the caches has to be as it was."""
        got = []
        for cache, before, which in ((self.k_cache, self.bytes[0], "k"), (self.v_cache, self.bytes[1], "v")):
            import torch
            raw = cache.contiguous().view(torch.uint8).cpu().numpy().reshape(-1)
            old = before.numpy().copy()
            if self.four:
                pools = [x.reshape(-1, self.Hkv, 9 * self.d) for x in (raw, old)]
                (c, s), (c0, s0) = (oracle.unpack_blocks(x, which) for x in pools)
                got.append((oracle.dequantise(c[self.row], s[self.row]), c[self.row], s[self.row]))
                c0[self.row], s0[self.row] = c[self.row], s[self.row]
                assert np.array_equal(c, c0) and np.array_equal(s, s0), "rows of others changed"
            else:
                a, b = (x.reshape(-1, self.Hkv * self.d * (1 if "kv" in self.dtype else 2)) for x in (raw, old))
                b[self.row] = a[self.row]
                assert np.array_equal(a, b), "rows of others changed"
                x = a[self.row].reshape(len(self.row), self.Hkv, -1)
                kind = "e4m3" if "kv" in self.dtype else self.dtype
                x = x if kind == "e4m3" else x.view(np.float16 if kind == "f16" else np.uint16)
                got.append((oracle.widen(x, kind), None, None))
        return got


def pair_size(y, n, interleaved):
    """|a| + |b| of the pair of every element (|y| where it does not rotate)."""
    m = np.abs(y)
    if n:
        m = m.copy()
        ia = 2 * np.arange(n) if interleaved else np.arange(n)
        ib = ia + (1 if interleaved else n)
        both = m[..., ia] + m[..., ib]
        m[..., ia] = m[..., ib] = both
    return m


def close(got, want, size, kind, mul=1.0):
    half, least = STEP[kind]
    want = want * mul
    if kind == "e4m3":
        want = np.clip(want, -448, 448)
    err = np.abs(got - want)
    bound = half * np.abs(want) * (1 + FP32) + least + 1.1 * FP32 * size * mul
    assert (err <= bound).all(), (err - bound).max()


def close_blocks(got, want, size, mul=1.0):
    """4-bit rows: every scale near max / 6, every code the nearest (or next to a border)."""
    y, codes, scales = got
    want, slack = want * mul, 2 * FP32 * size * mul
    s = oracle.widen(scales, "e4m3")
    amax = np.abs(want).reshape(*want.shape[:-1], -1, 16).max(-1)
    near = slack.reshape(*want.shape[:-1], -1, 16).max(-1)
    to = np.minimum(amax / 6, 448)
    assert (np.abs(s - to) <= 2.0 ** -4 * to * 1.001 + 2.0 ** -10 + near).all()
    s = np.repeat(s, 16, -1)
    mag = np.divide(np.abs(want), s, out=np.zeros_like(want), where=s > 0)
    half = np.where(mag < 2, 0.25, np.where(mag < 4, 0.5, np.where(mag < 6, 1.0, mag - 6 + 1e-12)))
    err = np.abs(y - want)
    assert (err <= np.where(s > 0, half * s, np.abs(want)) + slack).all()


DTYPES = ["f16", "bf16", "f16_e4m3kv", "f16_e2m1kv", "bf16_e2m1kv"]
# (d, Hq, Hkv, rot, interleaved, axes, norm, page): groups that are no power of two, odd head
# counts, partial and no rotation, every page size.
FORMS = [
    (128, 8, 2, 128, False, 1, True, 0), (128, 7, 7, 64, True, 1, False, 16), (64, 5, 1, 64, False, 3, True, 64),
    (64, 6, 3, 32, True, 2, True, 0), (128, 9, 3, 0, False, 1, True, 256), (128, 4, 1, 96, False, 4, False, 32),
    (128, 33, 11, 128, True, 3, True, 128), (64, 1, 1, 0, False, 1, False, 0),
]
# Ragged rows: none, one, the whole sequence, blocks cut at both ends, sequences without new rows.
SEQ = ([70, 0, 1, 33, 300, 16, 129], [69, 0, 0, 17, 250, 16, 100], [1, 0, 1, 16, 50, 0, 29])


@pytest.mark.parametrize("form", FORMS, ids=lambda f: "-".join(map(str, f)))
@pytest.mark.parametrize("dtype", DTYPES)
def test_append(fd, dtype, form):
    import torch
    d, Hq, Hkv, rot, inter, axes, norm, page = form
    s = Setup(fd, dtype, d, Hq, Hkv, *SEQ, page_size=page, seed=d + Hq + rot)
    T = s.rows.tokens
    inv = 10000.0 ** (-np.arange(rot // 2) / max(1, rot // 2))
    axis = [i % axes for i in range(rot // 2)] if axes > 1 else None
    rope = fd.Rope(inv, interleaved=inter, axes=axis, scale=0.75) if rot else None
    pos = s.pos[None]
    positions = None
    if axes > 1:
        pos = np.random.default_rng(rot).integers(-1000, 1 << 20, (rope.num_axes, T))
        positions = torch.tensor(pos, dtype=torch.int32).cuda()
    qw, kw = s.weights if norm else (None, None)
    offset = 1.0 if inter else 0.0
    k_out = torch.empty((T, Hkv, d), dtype=q_type(dtype), device="cuda")
    mul, v_mul = (0.5, 0.25) if "kv" in dtype else (1.0, 1.0)
    q = s.append(q_weight=qw, k_weight=kw, eps=1e-5, weight_offset=offset, rope=rope, positions=positions,
                 k_out=k_out, k_mul=mul, v_mul=v_mul)
    args = dict(offset=offset, eps=1e-5, norm=norm, inv_freq=inv, axes=axis, positions=pos,
                interleaved=inter, scale=0.75 if rot else 1.0)
    n16 = q_name(dtype)
    (kv, vv) = s.stored()
    for x, w, outs in ((s.q, qw, [q]), (s.k, kw, [k_out])):
        want, before = oracle.norm_rotate(f64(x), None if w is None else f64(w), **args)
        size = pair_size(before, rot // 2, inter)
        for o in outs:
            close(f64(o), want, size, n16)
    kind = {"f16": "f16", "bf16": "bf16", "f16_e4m3kv": "e4m3"}.get(dtype)
    v = f64(s.v)
    if kind:
        close(kv[0], want, size, kind, mul)
        close(vv[0], v, 0 * v, kind, v_mul)
    else:
        close_blocks(kv, want, size, mul)
        codes, scales = oracle.quantise(v * v_mul)      # v is exact until its one rounding
        assert np.array_equal(scales, vv[2])
        assert np.array_equal(oracle.dequantise(codes, scales), vv[0])


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("d,rot", [(64, 16), (64, 48), (128, 16), (128, 48), (128, 80), (128, 112)])
def test_partial_rotations_that_cut_blocks(fd, d, rot, inter):
    """Rotated parts that are no multiple of 32 (16-bit and E4M3 caches only)."""
    for dtype in ("bf16", "f16_e4m3kv"):
        test_append(fd, dtype, (d, 3, 3, rot, inter, 1, rot == 48, 0))
    s = Setup(fd, "f16_e2m1kv", d, 3, 3, [4], [0], [4])
    with pytest.raises(fd.FdError) as e:
        s.append(rope=fd.Rope([1.0] * (rot // 2)))
    assert e.value.status == fd.FD_ERR_UNSUPPORTED


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("d,page", [(64, 0), (128, 0), (64, 16), (128, 64)])
def test_gather_returns_what_is_stored(fd, dtype, d, page):
    """All rows, and a part of them: bit for bit the stored values."""
    s = Setup(fd, dtype, d, 4, 2, *SEQ, page_size=page, seed=3)
    s.append()
    want = [x[0] for x in s.stored()]
    k, v = s.rows.gather(s.k_cache, s.v_cache, block_table=s.table)
    assert np.array_equal(f64(k), want[0]) and np.array_equal(f64(v), want[1])
    # Every row of the sequences: the pattern the caches were filled with among them.
    every = fd.KVRows(4, 2, d, s.seqlens, dtype=dtype, page_size=page)
    k, v = every.gather(s.k_cache, s.v_cache, block_table=s.table)
    first = np.cumsum([0] + s.seqlens)
    idx = np.concatenate([first[b] + np.arange(s.begin[b], s.begin[b] + s.count[b]) for b in range(len(s.seqlens))])
    assert np.array_equal(f64(k)[idx], want[0]) and np.array_equal(f64(v)[idx], want[1])
    if s.four:
        at = s.place([0] * 7, s.seqlens)
        c, sc = oracle.unpack_blocks(s.k_cache.cpu().numpy().reshape(-1, 2, 9 * d), "k")
        assert np.array_equal(f64(k), oracle.dequantise(c, sc)[at], equal_nan=True)


def test_ties_and_saturation_are_exact(fd):
    """Rows of values on the borders between codes, against the oracle's ties to even."""
    import torch
    d = 64
    base = torch.tensor([6.0, 5, 3.5, 2.5, 1.75, 1.25, 0.75, 0.25, -5, -3.5, -2.5, -1.75, -1.25, -0.75, -0.25, 0])
    x = torch.stack([base.repeat(4) * m for m in (1.0, 0.125, 448.0, 600.0, 2.0 ** -9, 2.0 ** -10, 2.0 ** -12, 0.0)])
    for dtype in ("f16_e2m1kv", "bf16_e2m1kv"):
        k = x[:, None].to(q_type(dtype)).cuda()
        rows = fd.KVRows(1, 1, d, [8], dtype=dtype)
        kc, vc = (torch.zeros(fd.cache_shape(dtype, 1, d, [8]), dtype=torch.uint8, device="cuda") for _ in "kv")
        rows.append(None, k, k.clone(), kc, vc)
        codes, scales = oracle.quantise(f64(k))
        for cache, which in ((kc, "k"), (vc, "v")):
            c, s = oracle.unpack_blocks(cache.cpu().numpy(), which)
            assert np.array_equal(s[:8], scales)
            assert np.array_equal(oracle.dequantise(c, s)[:8], oracle.dequantise(codes, scales))
    k = torch.tensor([500.0, -1e4, 448, 464, 0.0009765625, 0.002, float("inf"), 17.0]).repeat(8).half()
    k = k[None, None].cuda()
    rows = fd.KVRows(1, 1, d, [1], dtype="f16_e4m3kv")
    kc, vc = (torch.zeros((1, 1, d), dtype=torch.uint8, device="cuda") for _ in "kv")
    rows.append(None, k, k.clone(), kc, vc)
    want = f64(k).clip(-448, 448)
    code = oracle.nearest_code(np.abs(want), ro.E4M3) + 128 * (want < 0)
    assert np.array_equal(kc.cpu().numpy(), code) and torch.equal(kc, vc)


def test_nan_and_infinity(fd):
    """A NaN stays in its own head (16 bits, norm), element (E4M3) or block of 16 (4 bits)."""
    import torch
    for dtype in DTYPES:
        k = torch.ones((2, 2, 128), dtype=q_type(dtype), device="cuda")
        k[0, 1, 37] = float("nan")
        k[1, 0, 5] = float("inf")
        rows = fd.KVRows(2, 2, 128, [2], dtype=dtype)
        kv = torch.uint8 if "kv" in dtype else k.dtype
        kc, vc = (torch.zeros(fd.cache_shape(dtype, 2, 128, [2]), dtype=kv, device="cuda") for _ in "kv")
        rows.append(None, k, k, kc, vc)
        for y in rows.gather(kc, vc):
            bad = np.zeros((2, 2, 128), dtype=bool)
            bad[0, 1, 32:48 if "e2m1" in dtype else 38] = True
            if "e2m1" not in dtype:
                bad[0, 1, 32:37] = False
            y = f64(y)
            assert np.array_equal(np.isnan(y), bad), dtype
            # 1 in 4 bits: 6 x E4M3(1 / 6) = 1.03125.
            one = oracle.dequantise(*oracle.quantise(np.ones(16)))[0] if "e2m1" in dtype else 1.0
            assert (y[0, 0] == one).all() and (y[1, 1] == one).all()
            top = {"f16_e4m3kv": 448.0, "f16_e2m1kv": 2688.0, "bf16_e2m1kv": 2688.0}.get(dtype, np.inf)
            assert y[1, 0, 5] == top
        q = rows.append(k, q_norm=True)
        assert np.isnan(f64(q)[0, 1]).all() and not np.isnan(f64(q)[0, 0]).any()


def test_zero_rows_and_norm_without_weights(fd):
    import torch
    x = torch.zeros((3, 4, 64), dtype=torch.float16, device="cuda")
    x[1] = 2.0
    rows = fd.KVRows(4, 4, 64, [3])
    y = f64(rows.append(x, q_norm=True, eps=1e-6))
    assert (y[0] == 0).all() and (y[1] == 1).all()
    # A weight without its norm switched on is not used.
    w = torch.full((64,), 3.0, dtype=torch.float16, device="cuda")
    assert torch.equal(rows.append(x, q_weight=w, q_norm=False), x)


def test_far_positions(fd):
    """int32's ends: the angle is as exact there as near zero."""
    import torch
    pos = np.array([0, 1, 10 ** 6, 2 ** 31 - 1, -2 ** 31, -12345678, 131071, 99999999])
    inv = 10000.0 ** (-np.arange(64) / 64)
    rows = fd.KVRows(2, 2, 128, [8])
    x = torch.randn((8, 2, 128), generator=torch.Generator().manual_seed(4)).half().cuda()
    # Frequencies that fp64 products keep exact: the oracle's angle is then the true one.
    inv = np.round(inv * 2 ** 20) / 2 ** 20
    y = rows.append(x, rope=fd.Rope(inv), positions=torch.tensor(pos, dtype=torch.int32).cuda())
    want, before = oracle.norm_rotate(f64(x), inv_freq=inv, positions=pos[None])
    close(f64(y), want, pair_size(before, 64, False), "f16")


def test_strides_and_in_place(fd):
    """Head-major and broadcast inputs, q and k in place, outputs without a cache."""
    import torch
    g = torch.Generator().manual_seed(9)
    d, H, T = 128, 3, 21
    rows = fd.KVRows(H, H, d, [30], [9], [T])
    inv = 10000.0 ** (-np.arange(64) / 64)
    rope = fd.Rope(inv)
    x = torch.randn((H, T, d), generator=g).half().cuda()
    k = torch.randn((1, H, d), generator=g).half().cuda()
    pos = np.arange(9, 30)[None]
    k_out = torch.empty((T, H, d), dtype=torch.float16, device="cuda")
    y = rows.append(x.transpose(0, 1), k.expand(T, H, d), k_out=k_out, rope=rope)
    for got, src in ((y, x.transpose(0, 1)), (k_out, k.expand(T, H, d))):
        want, before = oracle.norm_rotate(f64(src), inv_freq=inv, positions=pos)
        close(f64(got), want, pair_size(before, 64, False), "f16")
    q2, k2 = x.transpose(0, 1).contiguous(), k.expand(T, H, d).contiguous()
    rows.append(q2, k2, q_out=q2, k_out=k2, rope=rope)
    assert torch.equal(q2, y) and torch.equal(k2, k_out)
    with pytest.raises(ValueError):
        rows.append(torch.empty((T, H, 2 * d), dtype=torch.float16, device="cuda")[..., ::2])
    with pytest.raises(ValueError):
        rows.append(x.transpose(0, 1), q_out=x.transpose(0, 1))
    with pytest.raises(fd.FdError):                      # outputs over inputs
        rows.append(q2, k2, k_out=q2)


@pytest.mark.parametrize("dtype", ["bf16", "f16_e4m3kv", "f16_e2m1kv"])
def test_subsets_of_outputs(fd, dtype):
    """q alone, k alone, k in place while it is stored, and all together: the same values."""
    import torch
    s = Setup(fd, dtype, 64, 4, 2, [50, 7], [20, 0], [30, 7], page_size=32, seed=17)
    w = s.weights
    norm = dict(q_weight=w[0], k_weight=w[1], rope=fd.Rope(10000.0 ** (-np.arange(32) / 32)))
    k_out = torch.empty((37, 2, 64), dtype=q_type(dtype), device="cuda")
    q = s.append(k_out=k_out, **norm)
    kept = [x.clone() for x in (s.k_cache, s.v_cache)]
    s.stored()
    only = {n: x for n, x in norm.items() if n != "k_weight"}
    assert torch.equal(s.rows.append(s.q, **only), q)
    only = {n: x for n, x in norm.items() if n != "q_weight"}
    k2 = torch.empty_like(k_out)
    assert s.rows.append(None, s.k, k_out=k2, **only) is None
    assert torch.equal(k2, k_out)
    s.k_cache.zero_(), s.v_cache.zero_()
    k3 = s.k.contiguous()
    s.rows.append(None, k3, s.v, s.k_cache, s.v_cache, block_table=s.table, k_out=k3, **only)
    assert torch.equal(k3, k_out)
    got = s.rows.gather(s.k_cache, s.v_cache, block_table=s.table)
    want = s.rows.gather(*kept, block_table=s.table)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    # Without a cache a 4-bit handle rotates any multiple of 16.
    y = s.rows.append(s.q, rope=fd.Rope([0.5] * 8))
    ref, before = oracle.norm_rotate(f64(s.q), inv_freq=[0.5] * 8, positions=s.pos[None])
    close(f64(y), ref, pair_size(before, 8, False), q_name(dtype))


def test_bad_pages_are_reported_not_written(fd):
    import torch
    for dtype in DTYPES:
        s = Setup(fd, dtype, 64, 2, 2, [40, 40], [0, 0], [40, 40], page_size=16, seed=2)
        pages = s.k_cache.shape[0]
        s.table[0, 1], s.table[1, 2] = -1, pages
        keep = np.ones(80, dtype=bool)
        keep[16:32] = keep[72:80] = False
        s.row = s.row[keep]
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        q = s.append(status=status)
        assert status.item() == 1 and torch.equal(q, s.q)
        s.stored()                                        # nothing else was written
        status.zero_()
        k, v = s.rows.gather(s.k_cache, s.v_cache, block_table=s.table, status=status)
        assert status.item() == 1
        assert (f64(k)[~keep] == 0).all() and (f64(v)[~keep] == 0).all()
        good = s.table.clone()
        status.zero_()
        good[0, 1], good[1, 2] = 0, 1
        s.rows.gather(s.k_cache, s.v_cache, block_table=good, status=status)
        assert status.item() == 0


def test_offsets_past_32_bits(fd):
    """Pools of more than 2^32 bytes (and 2^32 half-bytes): the highest pages."""
    import torch
    for dtype, pages in (("f16", 9000), ("f16_e2m1kv", 32000)):
        d, H, page = 128, 8, 256
        shape = fd.cache_shape(dtype, H, d, None, pages, page)
        kv = torch.uint8 if "kv" in dtype else torch.float16
        kc, vc = (torch.empty(shape, dtype=kv, device="cuda") for _ in "kv")
        assert kc.numel() * kc.element_size() > 1 << 32
        table = torch.tensor([[pages - 1, pages // 2, 0]], dtype=torch.int32, device="cuda")
        rows = fd.KVRows(H, H, d, [600], dtype=dtype, page_size=page)
        g = torch.Generator().manual_seed(11)
        k, v = (torch.randn((600, H, d), generator=g).half().cuda() for _ in "kv")
        rows.append(None, k, v, kc, vc, block_table=table)
        got = rows.gather(kc, vc, block_table=table)
        for x, y in ((k, got[0]), (v, got[1])):
            want = f64(x)
            if "e2m1" in dtype:
                want = oracle.dequantise(*oracle.quantise(want))
            assert np.array_equal(f64(y), want)
        q = torch.randn((1, H, d), generator=g).half().cuda()
        out, lse = fd.Decoder(H, H, d, [600], [2], dtype, page_size=page).decode_paged(q, kc, vc, table)
        ref, ref_lse = oracle.decode_reference(f64(q), f64(got[0]), f64(got[1]), [600], "f64")
        assert np.abs(f64(out) - ref).max() <= 2e-3 and np.abs(f64(lse) - ref_lse).max() <= 1e-4


@pytest.mark.parametrize("dtype,page", [("f16", 0), ("bf16", 64), ("f16_e4m3kv", 16), ("f16_e2m1kv", 32),
                                        ("bf16_e2m1kv", 0)])
def test_prompt_then_tokens_then_decode(fd, dtype, page):
    """As they are used: a prompt appended in two parts, then token by token, a decode after each;
    the cache holds the oracle's rows and the decode is the oracle's over what is stored."""
    import torch
    Hq, Hkv, d = 8, 2, 128
    inv = 10000.0 ** (-np.arange(64) / 64)
    rope = fd.Rope(inv)
    g = torch.Generator().manual_seed(21)
    t16 = q_type(dtype)
    kv = torch.uint8 if "kv" in dtype else t16
    cap, pages = 128, 9
    table = torch.randperm(pages, generator=g)[:-(-cap // page)].int()[None].cuda() if page else None
    full = fd.cache_shape(dtype, Hkv, d, None, pages, page) if page else fd.cache_shape(dtype, Hkv, d, [cap])
    # Bytes that read as NaN in every type: nothing past the end may show.
    kc, vc = (torch.full(full, -1 if kv != torch.uint8 else 255, dtype=torch.int16 if kv != torch.uint8 else kv,
                         device="cuda").view(kv) for _ in "kv")
    clean = "e2m1" in dtype
    if not clean:
        kc.zero_(), vc.zero_()
    w = torch.linspace(0.5, 1.5, d).to(t16).cuda()
    L = 0
    for n in (37, 24, 1, 1, 1, 1):
        q, k, v = (torch.randn((n, h, d), generator=g).to(t16).cuda() for h in (Hq, Hkv, Hkv))
        L += n
        a = (kc, vc) if page else (kc[:fd.cache_shape(dtype, Hkv, d, [L])[0]], vc[:fd.cache_shape(dtype, Hkv, d, [L])[0]])
        rows = fd.KVRows(Hq, Hkv, d, [L], [L - n], [n], dtype, page)
        q = rows.append(q, k, v, *a, q_weight=w, k_weight=w, rope=rope, block_table=table)
        dec = fd.Decoder(Hq, Hkv, d, [L], [2], dtype, page_size=page)
        last = q[-1:].contiguous()
        out, lse = dec.decode_paged(last, *a, table) if page else dec(last, *a)
        gk, gv = fd.KVRows(Hq, Hkv, d, [L], dtype=dtype, page_size=page).gather(*a, block_table=table)
        ref, ref_lse = oracle.decode_reference(f64(last), f64(gk), f64(gv), [L], "f64")
        err = np.abs(f64(out) - ref)
        assert (err <= 2e-3 + (2.0 ** -8 if "bf16" in dtype else 0) * np.abs(ref)).all(), err.max()
        assert np.abs(f64(lse) - ref_lse).max() <= 1e-4


def test_streams_graph_and_two_calls_at_once(fd):
    """Calls on other streams, and a captured append, decode and gather replayed on new inputs."""
    import torch
    s = Setup(fd, "f16_e2m1kv", 128, 8, 2, [200, 90], [199, 89], [1, 1], page_size=64, seed=5)
    prefix = fd.KVRows(8, 2, 128, s.seqlens, dtype=s.dtype, page_size=64)
    g = torch.Generator().manual_seed(6)
    kv = torch.randn((2, 290, 2, 128), generator=g).half().cuda()
    prefix.append(None, kv[0], kv[1], s.k_cache, s.v_cache, block_table=s.table)
    dec = fd.Decoder(8, 2, 128, s.seqlens, [2, 2], s.dtype, page_size=64)
    rope = fd.Rope(10000.0 ** (-np.arange(64) / 64))

    def step(qkv):
        q = s.rows.append(qkv[:, :8], qkv[:, 8:10], qkv[:, 10:], s.k_cache, s.v_cache, rope=rope, block_table=s.table)
        out, lse = dec.decode_paged(q, s.k_cache, s.v_cache, s.table)
        return out, lse, prefix.gather(s.k_cache, s.v_cache, block_table=s.table)

    inputs = [torch.randn((2, 12, 128), generator=g).half().cuda() for _ in range(3)]
    want = []
    for x in inputs:
        out, lse, (k, v) = step(x)
        want.append((out.clone(), lse.clone(), k.clone(), v.clone()))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        out, lse, (k, v) = step(inputs[0])
    side.synchronize()
    assert torch.equal(out, want[0][0]) and torch.equal(k, want[0][2])
    static = inputs[0].clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(static)
    for x, w in zip(inputs, want):
        static.copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip((got[0], got[1], *got[2]), w):
            assert torch.equal(a, b)
    # Two appends and two gathers of different caches at once, on two streams.
    pair = [Setup(fd, "bf16_e2m1kv", 64, 4, 4, [500], [0], [500], seed=i) for i in (31, 32)]
    outs = [None, None]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for i in (0, 1):
        with torch.cuda.stream(streams[i]):
            pair[i].append()
            outs[i] = pair[i].rows.gather(pair[i].k_cache, pair[i].v_cache)
    torch.cuda.synchronize()
    for p, o in zip(pair, outs):
        assert np.array_equal(f64(o[1]), oracle.dequantise(*oracle.quantise(f64(p.v))))


def test_wrapper_checks(fd):
    import torch
    s = Setup(fd, "f16", 64, 4, 2, [20, 3], [19, 2], [1, 1], page_size=16)
    bad = [
        dict(q=s.q[:1]), dict(q=s.q.float()), dict(q=s.q.cpu()), dict(k=s.q), dict(v=s.v[..., :32]),
        dict(k_cache=s.k_cache[:, :8]), dict(v_cache=s.v_cache.bfloat16()), dict(v_cache=None),
        dict(block_table=None), dict(block_table=s.table.long()), dict(block_table=s.table[:1]),
        dict(block_table=s.table.cpu()), dict(q_weight=s.weights[0].float()),
        dict(positions=torch.zeros(2, dtype=torch.int32, device="cuda")),
        dict(status=torch.zeros(1, device="cuda")),
    ]
    good = dict(q=s.q, k=s.k, v=s.v, k_cache=s.k_cache, v_cache=s.v_cache, block_table=s.table)
    for change in bad:
        with pytest.raises(ValueError):
            s.rows.append(**{**good, **change})
    with pytest.raises(ValueError):
        s.rows.append(**good, rope=fd.Rope([1.0] * 16), positions=torch.zeros(3, dtype=torch.int32, device="cuda"))
    with pytest.raises(fd.FdError):                       # a table too narrow for the longest sequence
        s.rows.append(**{**good, "block_table": s.table[:, :1].contiguous()})
    s.append()
    s.stored()
    empty = fd.KVRows(4, 2, 64, [5, 0], [5, 0], [0, 0])
    out = empty.append(s.q[:0], s.k[:0], s.v[:0], torch.empty((5, 2, 64), dtype=torch.float16, device="cuda"),
                       torch.empty((5, 2, 64), dtype=torch.float16, device="cuda"))
    assert out.shape == (0, 4, 64)
