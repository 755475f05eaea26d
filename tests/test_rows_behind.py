"""What lies behind a sequence's last token (the next sequence of a contiguous cache, an earlier owner's
rows in its last page) has no part in its output, whatever it holds.

Tolerances: as in the older decode tests, out within 2e-3 (+ 2^-8 |out| for bf16's one rounding) and
lse within 1e-4 of the oracle.
"""
import numpy as np
import pytest

import oracle

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fd():
    import split_kv_flash_decode_gb300 as fd_mod
    from split_kv_flash_decode_gb300 import build
    build.build()
    return fd_mod


def f64(t):
    import torch
    return t.to(torch.float64).cpu().numpy()


def values(x, dtype):
    """Doubles of a cache tensor."""
    import torch
    return oracle.widen(x.cpu().numpy(), "e4m3") if x.dtype == torch.uint8 else f64(x)


def stored(x, dtype):
    import torch
    if dtype == "f16_e4m3kv":
        return x.to(torch.float8_e4m3fn).view(torch.uint8).cuda()
    return x.to(torch.float16 if dtype == "f16" else torch.bfloat16).cuda()


def check(out, lse, ref, ref_lse, dtype):
    err = np.abs(f64(out) - ref)
    assert (err <= 2e-3 + (2.0 ** -8 if dtype == "bf16" else 0) * np.abs(ref)).all(), np.nanmax(err)
    assert np.abs(f64(lse) - ref_lse).max() <= 1e-4


# (dtype, d, G, flag): every consumer of the split kernel.
FORMS = [("f16", 128, 1, 0), ("bf16", 64, 2, 0), ("f16", 64, 4, 0), ("f16", 128, 4, 0), ("bf16", 128, 4, 0),
         ("bf16", 64, 8, 0), ("f16", 128, 16, 0), ("f16", 128, 4, "FFMA"), ("bf16", 128, 8, "FFMA"),
         ("f16", 128, 4, "TCGEN05"), ("bf16", 128, 8, "TCGEN05"), ("f16", 128, 16, "TCGEN05"),
         ("f16_e4m3kv", 128, 4, 0), ("f16_e4m3kv", 128, 8, 0), ("f16_e4m3kv", 128, 16, 0)]
LENS = [1, 40, 15, 16, 17, 63, 64, 65, 127, 129, 500, 1030]
# What lies behind (E4M3 has no infinity).
CASES = [(f, bad) for f in FORMS for bad in ("nan", "inf", "-inf") if f[0] != "f16_e4m3kv" or bad == "nan"]


def case_id(x):
    return "-".join(map(str, x)) if isinstance(x, tuple) else str(x)


@pytest.mark.parametrize("form,bad", CASES, ids=case_id)
def test_contiguous_neighbours(fd, form, bad):
    """Every other sequence is NaN or infinite throughout; the ones between are as without them."""
    import torch
    dtype, d, G, flag = form
    g = torch.Generator().manual_seed(d + G)
    lens = [n for x in LENS for n in (x, 19)]
    N, Hkv = sum(lens), 2
    first = np.cumsum([0] + lens)
    x = torch.randn((2, N, Hkv, d), generator=g)
    for b in range(1, len(lens), 2):
        x[:, first[b]:first[b + 1]] = float(bad)
    k, v = (stored(y, dtype) for y in x)
    q = torch.randn((len(lens), G * Hkv, d), generator=g).to(torch.bfloat16 if dtype == "bf16" else torch.float16).cuda()
    flags = getattr(fd, "FD_PLAN_" + flag) if flag else 0
    for chunks in (0, 1):
        out, lse = fd.Decoder(G * Hkv, Hkv, d, lens, [2] * len(lens), dtype, flags, chunks)(q, k, v)
        good = list(range(0, len(lens), 2))
        keep = np.concatenate([np.arange(first[b], first[b + 1]) for b in good])
        ref, ref_lse = oracle.decode_reference(f64(q)[good], values(k, dtype)[keep], values(v, dtype)[keep], LENS, "f64")
        check(out[good], lse[good], ref, ref_lse, dtype)


@pytest.mark.parametrize("page", [16, 64, 256])
@pytest.mark.parametrize("form,bad", CASES, ids=case_id)
def test_last_pages(fd, form, page, bad):
    """Pools that hold NaN or infinities wherever no token of a sequence lies."""
    import torch
    dtype, d, G, flag = form
    g = torch.Generator().manual_seed(d + G + page)
    N, Hkv = sum(LENS), 2
    need = [-(-n // page) for n in LENS]
    perm = torch.randperm(sum(need) + 2, generator=g).int()
    table = torch.full((len(LENS), max(need)), int(perm[-1]), dtype=torch.int32)
    row, at = [], 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
        row += [int(table[b, r // page]) * page + r % page for r in range(LENS[b])]
    x = torch.randn((2, N, Hkv, d), generator=g)
    pools = []
    for y in x:
        pool = torch.full((len(perm) * page, Hkv, d), float(bad))
        pool[row] = y
        pools.append(stored(pool, dtype).view(len(perm), page, Hkv, d))
    q = torch.randn((len(LENS), G * Hkv, d), generator=g).to(torch.bfloat16 if dtype == "bf16" else torch.float16).cuda()
    ref, ref_lse = oracle.decode_reference(f64(q), values(stored(x[0], dtype), dtype), values(stored(x[1], dtype), dtype),
                                           LENS, "f64")
    flags = getattr(fd, "FD_PLAN_" + flag) if flag else 0
    dec = fd.Decoder(G * Hkv, Hkv, d, LENS, [2] * len(LENS), dtype, flags, page_size=page)
    out, lse = dec.decode_paged(q, *pools, table.cuda())
    assert dec.status() == fd.FD_OK
    check(out, lse, ref, ref_lse, dtype)


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f16_e4m3kv", "f16_e2m1kv", "bf16_e2m1kv"])
def test_recycled_page(fd, dtype):
    """A page that an earlier sequence's append left a NaN in, given to a new sequence of three tokens."""
    import torch
    Hkv, d, page = 2, 128, 64
    t16 = torch.bfloat16 if dtype.startswith("bf16") else torch.float16
    kv = torch.uint8 if "kv" in dtype else t16
    kc, vc = (torch.zeros(fd.cache_shape(dtype, Hkv, d, None, 3, page), dtype=kv, device="cuda") for _ in "kv")
    table = torch.tensor([[1]], dtype=torch.int32, device="cuda")
    g = torch.Generator().manual_seed(7)
    old = torch.randn((2, 64, Hkv, d), generator=g).to(t16).cuda()
    old[:, 5:] = float("nan")
    fd.KVRows(8, Hkv, d, [64], dtype=dtype, page_size=page).append(None, old[0], old[1], kc, vc, block_table=table)
    q, k, v = (torch.randn((3, h, d), generator=g).to(t16).cuda() for h in (8, Hkv, Hkv))
    rows = fd.KVRows(8, Hkv, d, [3], dtype=dtype, page_size=page)
    q = rows.append(q, k, v, kc, vc, block_table=table)
    out, lse = fd.Decoder(8, Hkv, d, [3], 1, dtype, page_size=page).decode_paged(q[-1:].contiguous(), kc, vc, table)
    k, v = rows.gather(kc, vc, block_table=table)
    ref, ref_lse = oracle.decode_reference(f64(q[-1:]), f64(k), f64(v), [3], "f64")
    err = np.abs(f64(out) - ref)
    # Weights of 4-bit and E4M3 caches are fp16: 2^-11 of values up to 8 in size.
    assert (err <= 4e-3 + (2.0 ** -8 if dtype.startswith("bf16") else 0) * np.abs(ref)).all()
    assert np.abs(f64(lse) - ref_lse).max() <= 1e-4
