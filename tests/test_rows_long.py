"""fd_append where a warp takes several rounds of head rows (prompts): against the oracle, with the
tolerances of test_rows.py, and bit for bit against the same tokens appended a few at a time, where every
warp takes one round.

A warp takes ceil(T (Hq + 2 Hkv) / 2432) head rows, rounded up to rounds of 512 / d: with 55 head rows at
d = 128, T = 400, 1000 and 3000 are 3, 6 and 14 rounds (all rows), at d = 64 2, 3 and 7.  33 q rows and 11 k
rows end in part rounds, and most warps cross from q to k or from k to v.
"""
import numpy as np
import pytest

import oracle
from test_rows import Setup, close, close_blocks, f64, fd, pair_size, q_name, q_type  # noqa: F401

pytestmark = pytest.mark.gpu

DTYPES = ["f16", "bf16", "f16_e4m3kv", "f16_e2m1kv", "bf16_e2m1kv"]
# (T, d, Hq, Hkv, rot, interleaved, norm, page)
FORMS = [(400, 128, 33, 11, 128, False, True, 0), (1000, 128, 33, 11, 64, True, True, 64),
         (3000, 128, 33, 11, 96, False, False, 0), (400, 64, 33, 11, 64, True, True, 16),
         (1000, 64, 33, 11, 32, False, True, 0), (3000, 64, 33, 11, 64, False, True, 256),
         (1500, 128, 5, 5, 0, False, True, 32)]


def lengths(T):
    """(seqlens, begin, count): T new tokens of ragged sequences, one without any."""
    count = [T // 2 + 3, 0, T // 3, 1]
    count.append(T - sum(count))
    begin = [17, 5, 0, 40, 1]
    return [a + n for a, n in zip(begin, count)], begin, count


@pytest.mark.parametrize("form", FORMS, ids=lambda f: "-".join(map(str, f)))
@pytest.mark.parametrize("dtype", DTYPES)
def test_prompts(fd, dtype, form):  # noqa: F811
    import torch
    T, d, Hq, Hkv, rot, inter, norm, page = form
    s = Setup(fd, dtype, d, Hq, Hkv, *lengths(T), page_size=page, seed=T + d)
    assert s.rows.tokens == T
    inv = 10000.0 ** (-np.arange(rot // 2) / max(1, rot // 2))
    rope = fd.Rope(inv, interleaved=inter) if rot else None
    qw, kw = s.weights if norm else (None, None)
    mul = 0.5 if "kv" in dtype else 1.0
    args = dict(q_weight=qw, k_weight=kw, eps=1e-5, rope=rope, k_mul=mul, v_mul=mul)
    k_out = torch.full((T, Hkv, d), 9.0, dtype=q_type(dtype), device="cuda")
    q = s.append(k_out=k_out, **args)
    kv, vv = s.stored()
    kept = [x.clone() for x in (s.k_cache, s.v_cache)]

    # The oracle.
    want = {}
    for name, x, w, out in (("q", s.q, qw, q), ("k", s.k, kw, k_out)):
        y, before = oracle.norm_rotate(f64(x), None if w is None else f64(w), eps=1e-5, norm=norm, inv_freq=inv,
                                       positions=s.pos[None], interleaved=inter)
        want[name] = (y, pair_size(before, rot // 2, inter))
        close(f64(out), *want[name], q_name(dtype))
    v = f64(s.v)
    kind = {"f16": "f16", "bf16": "bf16", "f16_e4m3kv": "e4m3"}.get(dtype)
    if kind:
        close(kv[0], *want["k"], kind, mul)
        close(vv[0], v, 0 * v, kind, mul)
    else:
        close_blocks(kv, *want["k"], mul)
        codes, scales = oracle.quantise(v * mul)
        assert np.array_equal(scales, vv[2]) and np.array_equal(oracle.dequantise(codes, scales), vv[0])

    # In place, into caches as they were before the call: the same bytes.
    s.k_cache.copy_(s.bytes[0].cuda().view(s.k_cache.dtype).view(s.k_cache.shape))
    s.v_cache.copy_(s.bytes[1].cuda().view(s.v_cache.dtype).view(s.v_cache.shape))
    q2, k2 = s.q.contiguous(), s.k.contiguous()
    s.rows.append(q2, k2, s.v, s.k_cache, s.v_cache, block_table=s.table, q_out=q2, k_out=k2, **args)
    same = lambda a, b: torch.equal(a.view(torch.uint8), b.view(torch.uint8))  # noqa: E731
    assert same(q2, q) and same(k2, k_out) and same(s.k_cache, kept[0]) and same(s.v_cache, kept[1])

    # A few tokens of each sequence at a time (one round a warp): the same bytes again.
    s.k_cache.copy_(s.bytes[0].cuda().view(s.k_cache.dtype).view(s.k_cache.shape))
    s.v_cache.copy_(s.bytes[1].cuda().view(s.v_cache.dtype).view(s.v_cache.shape))
    first = np.cumsum([0] + s.count)
    done = [0] * len(s.count)
    while done != s.count:
        n = [min(12, c - at) for c, at in zip(s.count, done)]
        rows = fd.KVRows(Hq, Hkv, d, s.seqlens, [a + at for a, at in zip(s.begin, done)], n, dtype, page)
        pick = torch.tensor(np.concatenate([np.arange(f + at, f + at + m) for f, at, m in zip(first, done, n)]),
                            device="cuda", dtype=torch.int64)
        part = rows.append(s.q[pick], s.k[pick], s.v[pick], s.k_cache, s.v_cache, block_table=s.table, **args)
        assert same(part, q[pick])
        done = [at + m for at, m in zip(done, n)]
    assert same(s.k_cache, kept[0]) and same(s.v_cache, kept[1])
