"""Cases and plain forms of the operators that fill, read back and attend over a KV cache.

append  per-head RMS norm of q and k, rotary positions (one axis or several, both pair
        orders) and the store of k and v into a contiguous or paged cache of 16-bit, FP8
        (E4M3) or 4-bit (E2M1 with one E4M3 scale per 16 values) elements: one launch.
gather  the rows of some sequences read back from such a cache into contiguous 16-bit
        tensors, as prefill attention over an earlier prefix needs them.
chunk   append into a 4-bit cache, then gather of the whole sequences (chunked prefill).
decode  split-KV attention of one query token per sequence over a 4-bit cache.

``run`` computes the plain form in 32-bit torch operations, or, where ``own`` is true, makes
the framework's calls.  Byte layout of a 4-bit cache (16 tokens x one KV head = one block of
9 d bytes): see ``_unpack_k`` and ``_unpack_v``.
"""
import math
import random

import torch

own = False

_Q = {"f16": torch.float16, "bf16": torch.bfloat16, "f16_e4m3kv": torch.float16,
      "f16_e2m1kv": torch.float16, "bf16_e2m1kv": torch.bfloat16}
_E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def listed():
    return [
        # One new token of one conversation: the latency of a decode step's first kernel.
        dict(name="append_one", op="append", B=1, L=4097, n=1, Hq=32, Hkv=8, d=128, dtype="f16",
             page=64, mix=0, norm=True, rot=128, inter=False, axes=1),
        # A decode step of a ragged serving batch over an FP8 cache in small pages.
        dict(name="append_step_fp8", op="append", B=64, L=1024, n=1, Hq=32, Hkv=8, d=128,
             dtype="f16_e4m3kv", page=16, mix=5, norm=False, rot=64, inter=True, axes=1),
        # Ragged prompts with image positions (three axes) into a contiguous cache.
        dict(name="append_prompts_3axes", op="append", B=5, L=2048, n=2048, Hq=32, Hkv=4, d=128,
             dtype="bf16", page=0, mix=9, norm=True, rot=128, inter=False, axes=3),
        # Long prompts: the largest append.
        dict(name="append_prompts_32k", op="append", B=8, L=4096, n=4096, Hq=32, Hkv=8, d=128,
             dtype="f16", page=64, mix=0, norm=True, rot=128, inter=False, axes=1),
        # Chunked prefill over a 4-bit cache: 512 new tokens, then K and V of all 8K tokens.
        dict(name="chunk_4bit", op="chunk", B=1, L=8192, n=512, Hq=32, Hkv=8, d=128,
             dtype="f16_e2m1kv", page=128, mix=0),
        # Prefix reuse: ragged prefixes read back from an FP8 cache.
        dict(name="gather_fp8_ragged", op="gather", B=13, L=4096, Hq=32, Hkv=8, d=128,
             dtype="f16_e4m3kv", page=32, mix=3),
        # One long prefix read back from a 4-bit cache.
        dict(name="gather_4bit_32k", op="gather", B=1, L=32768, Hq=32, Hkv=8, d=128,
             dtype="bf16_e2m1kv", page=0, mix=0),
        # The smallest decode: two short conversations, one query head per KV head.
        dict(name="decode_short_g1", op="decode", B=2, L=517, Hq=8, Hkv=8, d=64, dtype="f16_e2m1kv",
             page=0, mix=0, W=4),
        # One 32K conversation.
        dict(name="decode_32k_g4", op="decode", B=1, L=32768, Hq=32, Hkv=8, d=128,
             dtype="f16_e2m1kv", page=0, mix=0, W=8),
        # Ragged paged batch, with empty and one-token sequences.
        dict(name="decode_ragged_g16", op="decode", B=17, L=16384, Hq=64, Hkv=4, d=128,
             dtype="bf16_e2m1kv", page=64, mix=7, W=4),
        # One 128K conversation.
        dict(name="decode_128k_g8", op="decode", B=1, L=131072, Hq=64, Hkv=8, d=128,
             dtype="f16_e2m1kv", page=0, mix=0, W=8),
        # The full serving batch: 64 conversations of 8K tokens.
        dict(name="decode_64x8k_g4", op="decode", B=64, L=8192, Hq=32, Hkv=8, d=128,
             dtype="bf16_e2m1kv", page=0, mix=0, W=16),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["append", "append", "chunk", "gather", "decode", "decode", "decode"])
    d, Hkv = rng.choice([64, 128, 128]), rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 2, 4, 8, 16])
    c = dict(op=op, B=_log(rng, 1, 64), Hq=G * Hkv, Hkv=Hkv, d=d,
             page=rng.choice([0, 16, 32, 64, 128, 256]), mix=rng.choice([0, rng.randrange(1, 1000)]))
    most = 400000 // (c["B"] * Hkv)          # tokens x KV heads of a drawn case stay below this
    c["L"] = _log(rng, 1, max(1, min(40000, most)))
    if op == "append":
        c["L"] = min(c["L"], max(1, 250000 // (c["B"] * Hkv * (G + 2))))
        c["dtype"] = rng.choice(["f16", "bf16", "f16_e4m3kv"])
        c["n"] = rng.choice([1, _log(rng, 1, c["L"])])
        c["norm"], c["inter"] = rng.random() < 0.5, rng.random() < 0.4
        c["rot"] = 16 * rng.randrange(0, d // 16 + 1)
        c["axes"] = rng.choice([1, 1, 2, 3]) if c["rot"] else 1
    elif op == "chunk":
        c["dtype"] = rng.choice(["f16_e2m1kv", "bf16_e2m1kv"])
        c["n"] = _log(rng, 1, c["L"])
    elif op == "gather":
        c["dtype"] = rng.choice(["f16", "bf16", "f16_e4m3kv", "f16_e2m1kv", "bf16_e2m1kv"])
    else:
        c["dtype"] = rng.choice(["f16_e2m1kv", "bf16_e2m1kv"])
        c["W"] = _log(rng, 1, 16)
    return c


# ------------------------------------------------------------------ shapes of a case

def _lengths(case):
    """Tokens of each sequence after the call: equal, or ragged with an empty and a one-token one."""
    B, L = case["B"], case["L"]
    if not case["mix"]:
        return [L] * B
    r = random.Random(case["mix"])
    lens = [L, 0, 1][:B] + [_log(r, 1, L) for _ in range(B - 3)]
    r.shuffle(lens)
    return lens


def _news(case, lens):
    """New tokens of each sequence: the last ones of it."""
    if not case["mix"]:
        return [min(case["n"], x) for x in lens]
    r = random.Random(case["mix"] + 1)
    return [min(x, case["n"] if r.random() < 0.7 else r.randrange(0, case["n"] + 1)) for x in lens]


def _four(case):
    return "e2m1" in case["dtype"]


def _blocks(case, lens):
    """Rows of 16 tokens (4-bit) of a contiguous cache: every sequence starts a new one."""
    return [-(-x // 16) for x in lens]


def _row_bytes(case):
    """Bytes of one (token, KV head) of K or of V."""
    return case["d"] * 9 / 16 if _four(case) else case["d"] * (1 if "e4m3" in case["dtype"] else 2)


def work(case):
    lens = _lengths(case)
    N, Hq, Hkv, d = sum(lens), case["Hq"], case["Hkv"], case["d"]
    row = Hkv * _row_bytes(case)
    if case["op"] == "append":
        T = sum(_news(case, lens))
        per = 2 * 2 * Hq * d + 2 * 2 * Hkv * d + 2 * row + 4 * case["axes"] * (case["axes"] > 1)
        return {"bytes": max(1, T * per), "flops": T * (Hq + Hkv) * (3 * case["rot"] + 4 * d * case["norm"])}
    if case["op"] == "chunk":
        T = sum(_news(case, lens))
        return {"bytes": max(1, T * (2 * 2 * Hkv * d + 2 * row) + N * (2 * row + 2 * 2 * Hkv * d)), "flops": 0}
    if case["op"] == "gather":
        return {"bytes": max(1, N * (2 * row + 2 * 2 * Hkv * d)), "flops": 0}
    return {"bytes": N * 2 * row + case["B"] * Hq * (2 * 2 * d + 4), "flops": 4 * N * Hq * d}


# ------------------------------------------------------------------ 4-bit blocks in plain torch

def _quantise(x):
    """Codes (E2M1, sign in bit 3) and E4M3 scales of the blocks of 16 along the last axis: the
    scale is max|x| / 6 and a code x / scale, each to the nearest, ties to even."""
    y = x.unflatten(-1, (-1, 16))
    s8 = (y.abs().amax(-1) / 6).clamp(max=448).to(torch.float8_e4m3fn)
    s = s8.to(x.dtype).unsqueeze(-1)
    m = torch.where(s > 0, y.abs() / s, torch.zeros_like(y))
    c = ((m > 0.25).to(torch.uint8) + (m >= 0.75) + (m > 1.25) + (m >= 1.75) + (m > 2.5) + (m >= 3.5)
         + (m > 5))
    return (c + 8 * torch.signbit(y)).to(torch.uint8).flatten(-2), s8


def _values(codes, s8):
    lut = torch.tensor(_E2M1 + [-x for x in _E2M1], device=codes.device)
    y = lut[codes.long()].unflatten(-1, (-1, 16)) * s8.float().unsqueeze(-1)
    return y.flatten(-2)


def _nibbles(b):
    return torch.stack((b & 15, b >> 4), -1).flatten(-2)


def _bytes(c):
    return c[..., 0::2] | (c[..., 1::2] << 4)


def _swap(x, d):
    """Groups 1, 3, 5, 7 (d = 128) or 2, 3, 6, 7 (d = 64) of [..., 8 groups, 8 token pairs, 2, :]
    hold their upper four token pairs first."""
    odd = torch.arange(8, device=x.device) // (1 if d == 128 else 2) % 2 == 1
    return torch.where(odd[:, None, None, None], x.roll(4, -3), x)


def _pack_k(codes, s8):
    """K block from codes [..., 16, d], scales [..., 16, d / 16]: 16 rows of d / 2 bytes (even
    element in the low half), then 16 rows of scales."""
    return torch.cat((_bytes(codes).flatten(-2), s8.view(torch.uint8).flatten(-2)), -1)


def _pack_v(codes, s8):
    """V block: 8 groups of d / 8 elements, each [8 token pairs][2 tokens][d / 16 bytes] with the
    pairs in the order of ``_swap``; then the scales, [d / 16][16 tokens]."""
    d = codes.shape[-1]
    g = _bytes(codes).unflatten(-1, (8, d // 16)).movedim(-2, -3).unflatten(-2, (8, 2))
    return torch.cat((_swap(g, d).flatten(-4), s8.view(torch.uint8).mT.flatten(-2)), -1)


def _unpack_k(pool, d):
    """Values [blocks, Hkv, 16, d] of K blocks [blocks, Hkv, 9 d]."""
    return _values(_nibbles(pool[..., :8 * d].unflatten(-1, (16, d // 2))),
                   pool[..., 8 * d:].unflatten(-1, (16, d // 16)).view(torch.float8_e4m3fn))


def _unpack_v(pool, d):
    g = _swap(pool[..., :8 * d].unflatten(-1, (8, 8, 2, d // 16)), d).flatten(-3, -2)
    return _values(_nibbles(g.movedim(-3, -2).flatten(-2)),
                   pool[..., 8 * d:].unflatten(-1, (d // 16, 16)).mT.contiguous().view(torch.float8_e4m3fn))


# ------------------------------------------------------------------ inputs

def _rope_host(case):
    """Frequencies (radians a position) and the axis of each pair: sections in turn, as image
    models cut their pairs."""
    half = case["rot"] // 2
    inv = [10000.0 ** (-i / half) for i in range(half)]
    cuts = [half * (a + 1) // case["axes"] for a in range(case["axes"])]
    return inv, [sum(i >= c for c in cuts) for i in range(half)]


def _fill(case, pack, nrows, dev, gen, amp):
    """A cache of `nrows` rows (tokens, or blocks of 16 tokens) as earlier appends left it, its
    channels of sizes `amp`; `pack` lays out a 4-bit one."""
    H, d = case["Hkv"], case["d"]
    if not _four(case):
        x = torch.randn((nrows, H, d), device=dev, generator=gen)
        if "e4m3" in case["dtype"]:
            return (x * amp).to(torch.float8_e4m3fn).view(torch.uint8)
        return (x * amp).to(_Q[case["dtype"]])
    out = torch.empty((nrows, H, 9 * d), dtype=torch.uint8, device=dev)
    step = max(1, (1 << 25) // (16 * H * d))
    for a in range(0, nrows, step):
        n = min(step, nrows - a)
        out[a:a + n] = pack(*_quantise(torch.randn((n, H, 16, d), device=dev, generator=gen) * amp))
    return out


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    lens, Hq, Hkv, d, page = _lengths(case), case["Hq"], case["Hkv"], case["d"], case["page"]
    s = {"case": case, "lens": lens}
    unit = 16 if _four(case) else 1                       # tokens a cache row
    if page:
        need = [-(-x // page) for x in lens]
        pages = sum(need) + 3
        perm = torch.randperm(pages, device=dev, generator=gen).to(torch.int32)
        table = torch.zeros((case["B"], max(1, max(need))), dtype=torch.int32, device=dev)
        at = 0
        for b, n in enumerate(need):
            table[b, :n] = perm[at:at + n]
            at += n
        nrows, s["table"] = pages * page // unit, table
    else:
        nrows, s["table"] = (sum(_blocks(case, lens)) if _four(case) else sum(lens)), None
        nrows = max(1, nrows)
        n = torch.tensor([16 * x for x in _blocks(case, lens)] if _four(case) else lens, device=dev)
        s["first"] = torch.cumsum(n, 0) - n               # cache row of each sequence's first token
    # Keys have channels of different sizes; values do not.
    amp = torch.rand(d, device=dev, generator=gen) * 1.5 + 0.25
    pools = [_fill(case, _pack_k, nrows, dev, gen, amp), _fill(case, _pack_v, nrows, dev, gen, 1.0)]
    if page:
        pools = [x.view(pages, page // unit, *x.shape[1:]) for x in pools]
    s["k_cache"], s["v_cache"] = pools
    q_type = _Q[case["dtype"]]
    normal = lambda *shape: torch.randn(shape, device=dev, generator=gen)  # noqa: E731
    if case["op"] in ("append", "chunk"):
        new = _news(case, lens)
        T = sum(new)
        # One projection gives q, k and v side by side: the operators read them in place.
        qkv = (normal(T, Hq + 2 * Hkv, d)).to(q_type)
        s["q"], s["k"], s["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        s["begin"], s["new"] = [x - n for x, n in zip(lens, new)], new
        s["sid"], s["row"] = _tokens(s["begin"], new, dev)
    if case["op"] == "append":
        s["q_weight"] = (1 + 0.2 * normal(d)).to(q_type) if case["norm"] else None
        s["k_weight"] = (1 + 0.2 * normal(d)).to(q_type) if case["norm"] else None
        s["inv"], s["axis"] = _rope_host(case)
        s["inv_device"] = torch.tensor(s["inv"], dtype=torch.float64, device=dev)
        s["axis_device"] = torch.tensor(s["axis"], device=dev, dtype=torch.int64)
        s["positions"] = None
        if case["axes"] > 1:
            # Text and image positions: near each other, far from zero now and then.
            base = torch.randint(0, 1 << 17, (1, T), device=dev, generator=gen)
            s["positions"] = (base + torch.randint(0, 64, (case["axes"], T), device=dev,
                                                   generator=gen)).to(torch.int32)
    if case["op"] == "decode":
        s["q"] = normal(case["B"], Hq, d).to(q_type)
    if case["op"] in ("chunk", "gather", "decode"):
        s["all_sid"], s["all_row"] = _tokens([0] * case["B"], lens, dev)
    s["kept"] = {}                                        # the framework's plans, made at the first call
    return s


def _tokens(begin, count, dev):
    """Sequence and row (within it) of every token of the given ranges."""
    n = torch.tensor(count, device=dev)
    sid = torch.repeat_interleave(torch.arange(len(count), device=dev), n)
    first = torch.cumsum(n, 0) - n - torch.tensor(begin, device=dev)
    return sid, torch.arange(sid.numel(), device=dev) - first[sid]


# ------------------------------------------------------------------ plain forms

def _pool_rows(s, sid, row):
    """Row of the cache, taken as [rows, Hkv, d], of each (sequence, row)."""
    if s["table"] is not None:
        page = s["case"]["page"]
        return s["table"][sid, row // page].long() * page + row % page
    return s["first"][sid] + row


def _cache_values(s):
    """K and V of the whole cache in 32 bits, [rows, Hkv, d]."""
    case, d = s["case"], s["case"]["d"]
    if _four(case):
        k = _unpack_k(s["k_cache"].view(-1, case["Hkv"], 9 * d), d).transpose(1, 2)
        v = _unpack_v(s["v_cache"].view(-1, case["Hkv"], 9 * d), d).transpose(1, 2)
        return k.flatten(0, 1), v.flatten(0, 1)
    t = torch.float8_e4m3fn if "e4m3" in case["dtype"] else _Q[case["dtype"]]
    return tuple(s[n].view(t).view(-1, case["Hkv"], d).float() for n in ("k_cache", "v_cache"))


def _norm_rotate(x, weight, s):
    """RMS norm of each head, then the rotation of its first `rot` elements."""
    case = s["case"]
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * weight.float()
    rot = case["rot"]
    if not rot:
        return x
    pos = s["positions"] if s["positions"] is not None else s["row"][None]
    angle = pos[s["axis_device"]].double().T * s["inv_device"]
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    if case["inter"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y = torch.cat((a * cos - b * sin, a * sin + b * cos), -1)
    return torch.cat((y, x[..., rot:]), -1)


def _plain_append(s):
    case = s["case"]
    t = _Q[case["dtype"]]
    q = _norm_rotate(s["q"], s["q_weight"], s).to(t)
    k, v = _norm_rotate(s["k"], s["k_weight"], s), s["v"].float()
    at = _pool_rows(s, s["sid"], s["row"])
    for name, x in (("k_cache", k), ("v_cache", v)):
        pool = s[name].view(-1, case["Hkv"], case["d"])
        if "e4m3" in case["dtype"]:
            pool[at] = x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        else:
            pool[at] = x.to(t)
    return {"q": q, "k_cache": _seen(s, "k_cache"), "v_cache": _seen(s, "v_cache")}


def _seen(s, name):
    """The whole cache as the numbers it holds."""
    return s[name].view(torch.float8_e4m3fn) if "e4m3" in s["case"]["dtype"] else s[name]


def _plain_gather(s):
    """Chunk and gather: the rows of every sequence, those appended now among them."""
    case = s["case"]
    t = _Q[case["dtype"]]
    at = _pool_rows(s, s["all_sid"], s["all_row"])
    k, v = _cache_values(s)
    if case["op"] == "chunk":
        to = _pool_rows(s, s["sid"], s["row"])
        k, v = k.contiguous(), v.contiguous()
        k[to] = _values(*_quantise(s["k"].float()))
        v[to] = _values(*_quantise(s["v"].float()))
    return {"k": k[at].to(t), "v": v[at].to(t)}


def _plain_decode(s):
    case, lens = s["case"], s["lens"]
    B, Hq, Hkv, d = case["B"], case["Hq"], case["Hkv"], case["d"]
    top = max(1, max(lens))
    row = torch.arange(top, device=s["q"].device).expand(B, top)
    there = row < torch.tensor(lens, device=row.device)[:, None]
    at = _pool_rows(s, torch.arange(B, device=row.device)[:, None], row * there)
    k, v = _cache_values(s)
    at = at.clamp(max=k.shape[0] - 1)                     # sequences without a token at the end
    k, v = k[at].transpose(1, 2), v[at].transpose(1, 2)   # [B, Hkv, top, d]
    q = s["q"].float().unflatten(1, (Hkv, Hq // Hkv))
    x = (q @ k.mT) / math.sqrt(d)
    x = x.masked_fill(~there[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = torch.exp(x - m)
    l = p.sum(-1, keepdim=True)
    out = torch.where(l > 0, (p @ v) / l, torch.zeros_like(q))
    lse = (m + torch.log(l)).view(B, Hq)
    return {"out": out.reshape(B, Hq, d).to(_Q[case["dtype"]]), "lse": lse}


# ------------------------------------------------------------------ the framework's calls

def _plan(s, what):
    """Plans hold host memory only and serve every call of the same lengths."""
    import split_kv_flash_decode_gb300 as fd
    case = s["case"]
    if what not in s["kept"]:
        if what == "decode":
            s["kept"][what] = fd.Decoder(case["Hq"], case["Hkv"], case["d"], s["lens"], [case["W"]] * case["B"],
                                         case["dtype"], page_size=case["page"])
        else:
            new = what == "new"
            s["kept"][what] = fd.KVRows(case["Hq"], case["Hkv"], case["d"], s["lens"], s["begin"] if new else None,
                                        s["new"] if new else None, dtype=case["dtype"], page_size=case["page"])
        if case["op"] == "append" and case["rot"]:
            s["kept"]["rope"] = fd.Rope(s["inv"], interleaved=case["inter"], axes=s["axis"])
    return s["kept"][what]


def _own(s):
    case = s["case"]
    if case["op"] == "append":
        q = _plan(s, "new").append(s["q"], s["k"], s["v"], s["k_cache"], s["v_cache"],
                                   q_weight=s["q_weight"], k_weight=s["k_weight"], eps=1e-6,
                                   rope=s["kept"].get("rope"), positions=s["positions"],
                                   block_table=s["table"])
        return {"q": q, "k_cache": _seen(s, "k_cache"), "v_cache": _seen(s, "v_cache")}
    if case["op"] == "decode":
        dec = _plan(s, "decode")
        if s["table"] is None:
            out, lse = dec(s["q"], s["k_cache"], s["v_cache"])
        else:
            out, lse = dec.decode_paged(s["q"], s["k_cache"], s["v_cache"], s["table"])
        return {"out": out, "lse": lse}
    if case["op"] == "chunk":
        _plan(s, "new").append(None, s["k"], s["v"], s["k_cache"], s["v_cache"], block_table=s["table"])
    k, v = _plan(s, "all").gather(s["k_cache"], s["v_cache"], block_table=s["table"])
    return {"k": k, "v": v}


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    return _plain_append(state) if op == "append" else _plain_decode(state) if op == "decode" \
        else _plain_gather(state)


# ------------------------------------------------------------------ 64 bits, written apart

def _exact_blocks(pool, which, d):
    """Doubles [tokens, Hkv, d] of 4-bit blocks, by the byte offset of every (token, element)."""
    NB, H = pool.shape[0], pool.shape[1]
    tok, el = torch.meshgrid(torch.arange(16), torch.arange(d), indexing="ij")
    if which == "k":
        byte, scale = tok * (d // 2) + el // 2, 8 * d + tok * (d // 16) + el // 16
    else:
        g = el // (d // 8)
        pair = (tok // 2) ^ (4 * ((g if d == 128 else g // 2) % 2))
        byte = g * d + pair * (d // 8) + (tok % 2) * (d // 16) + (el % (d // 8)) // 2
        scale = 8 * d + (el // 16) * 16 + tok
    dev = pool.device
    x = pool[:, :, byte.flatten().to(dev)].to(torch.int16)
    x = torch.where((el.flatten() % 2 == 1).to(dev), x // 16, x % 16)
    e, m = (x % 8) // 2, x % 2
    mag = torch.where(e == 0, 0.5 * m, (1 + 0.5 * m) * torch.exp2(e.double() - 1))
    z = pool[:, :, scale.flatten().to(dev)].to(torch.int16)
    se, sm = (z // 8) % 16, z % 8
    sc = torch.where(se == 0, sm / 512.0, (1 + sm / 8.0) * torch.exp2(se.double() - 7))
    y = torch.where(x >= 8, -mag, mag) * torch.where(z >= 128, -sc, sc)
    return y.view(NB, H, 16, d).permute(0, 2, 1, 3).reshape(NB * 16, H, d)


def _exact_index(s, b, lo, hi):
    """Cache rows of tokens lo .. hi - 1 of sequence b."""
    case = s["case"]
    if s["table"] is None:
        per = [16 * x for x in _blocks(case, s["lens"])] if _four(case) else s["lens"]
        return torch.arange(lo, hi, device="cuda") + sum(per[:b])
    t = torch.arange(lo, hi, device="cuda")
    return s["table"][b].long()[t // case["page"]] * case["page"] + t % case["page"]


def _exact_cache(s, name, rows):
    """Doubles of the given cache rows."""
    case, d, H = s["case"], s["case"]["d"], s["case"]["Hkv"]
    if _four(case):
        pool = s[name].view(-1, H, 9 * d)
        blocks, at = torch.unique(rows // 16, return_inverse=True)
        y = torch.empty((rows.numel(), H, d), dtype=torch.float64, device="cuda")
        step = max(1, (1 << 24) // (16 * H * d))
        vals = [_exact_blocks(pool[blocks[i:i + step]], name[0], d) for i in range(0, blocks.numel(), step)]
        if vals:
            y = torch.cat(vals)[at * 16 + rows % 16]
        return y
    t = torch.float8_e4m3fn if "e4m3" in case["dtype"] else _Q[case["dtype"]]
    return s[name].view(-1, H, d)[rows].view(t).double()


def _exact_code(x):
    """Nearest stored value of every element (blocks of 16 on the last axis), ties to even."""
    grid = torch.tensor(_E2M1, dtype=torch.float64, device=x.device)
    y = x.unflatten(-1, (-1, 16))
    s = (y.abs().amax(-1, keepdim=True) / 6).clamp(max=448).float().to(torch.float8_e4m3fn).double()
    m = y.abs() / torch.where(s > 0, s, torch.ones_like(s)) * (s > 0)
    hi = torch.searchsorted(grid, m.contiguous()).clamp(max=7)
    lo = (hi - 1).clamp(min=0)
    down, up = m - grid[lo], grid[hi] - m
    best = torch.where((down < up) | ((down == up) & (lo % 2 == 0)), lo, hi)
    return (grid[best] * torch.sign(y) * s).flatten(-2)


def exact(case, seed):
    s = prepare(case, seed)
    lens, d, Hkv = s["lens"], case["d"], case["Hkv"]
    if case["op"] == "append":
        eps = 1e-6
        pos = s["positions"].double() if s["positions"] is not None else s["row"].double()[None]
        turn = torch.zeros((s["row"].numel(), case["rot"] // 2), dtype=torch.float64, device="cuda")
        for i, f in enumerate(s["inv"]):
            turn[:, i] = pos[s["axis"][i]] * f
        unit = torch.polar(torch.ones_like(turn), turn)[:, None]
        done = []
        for x, w in ((s["q"], s["q_weight"]), (s["k"], s["k_weight"])):
            y = x.double()
            if w is not None:
                y = y / torch.sqrt((y * y).sum(-1, keepdim=True) / d + eps) * w.double()
            r, h = case["rot"], case["rot"] // 2
            z = (torch.complex(y[..., 0:r:2].contiguous(), y[..., 1:r:2].contiguous()) if case["inter"]
                 else torch.complex(y[..., :h].contiguous(), y[..., h:r].contiguous())) * unit
            z = torch.view_as_real(z)
            y[..., :r] = z.flatten(-2) if case["inter"] else torch.cat((z[..., 0], z[..., 1]), -1)
            done.append(y)
        caches = []
        rows = torch.cat([_exact_index(s, b, s["begin"][b], lens[b]) for b in range(case["B"])])
        t = torch.float8_e4m3fn if "e4m3" in case["dtype"] else _Q[case["dtype"]]
        for name, x in (("k_cache", done[1]), ("v_cache", s["v"].double())):
            pool = s[name].view(t).double()
            pool.view(-1, Hkv, d)[rows] = x
            caches.append(pool)
        return {"q": done[0], "k_cache": caches[0], "v_cache": caches[1]}
    if case["op"] in ("chunk", "gather"):
        rows = torch.cat([_exact_index(s, b, 0, lens[b]) for b in range(case["B"])])
        got = {"k": _exact_cache(s, "k_cache", rows), "v": _exact_cache(s, "v_cache", rows)}
        if case["op"] == "chunk":
            start, at = 0, 0
            for b in range(case["B"]):
                n = s["new"][b]
                for name in ("k", "v"):
                    got[name][start + s["begin"][b]:start + lens[b]] = _exact_code(s[name][at:at + n].double())
                start, at = start + lens[b], at + n
        return got
    G = case["Hq"] // Hkv
    out = torch.zeros((case["B"], case["Hq"], d), dtype=torch.float64, device="cuda")
    lse = torch.full((case["B"], case["Hq"]), -math.inf, dtype=torch.float64, device="cuda")
    for b in range(case["B"]):
        if lens[b] == 0:
            continue
        rows = _exact_index(s, b, 0, lens[b])
        k, v = _exact_cache(s, "k_cache", rows), _exact_cache(s, "v_cache", rows)
        q = s["q"][b].double().view(Hkv, G, d)
        x = torch.einsum("hgd,lhd->hgl", q, k) / d ** 0.5
        lse[b] = torch.logsumexp(x, -1).flatten()
        out[b] = torch.einsum("hgl,lhd->hgd", torch.softmax(x, -1), v).reshape(case["Hq"], d)
    return {"out": out, "lse": lse}
