"""Cases and plain forms of the operators of a step of speculative decoding over a KV cache.

attend  attention of all drafted tokens of every sequence (a chain, or a tree given by one mask of
        64 bits per token) over a contiguous or paged cache of 16-bit, FP8 (E4M3) or 4-bit (E2M1 with
        one E4M3 scale per 16 values) elements, whose last rows hold the drafted tokens.
verify  which drafted tokens stand, and the token that follows them, from the target's
        probabilities and given random numbers: trees of given tokens, or chains with the
        probabilities that their tokens were drawn from.
keep    the accepted tokens' rows moved to the front of the drafted ones, in place.

``run`` computes the plain form, or, where ``own`` is true, makes the framework's calls.
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
        # The smallest: a chain of four over one short conversation, one query head per KV head.
        dict(name="attend_short_chain", op="attend", B=1, L=517, n=4, tree=False, Hq=8, Hkv=8, d=64,
             dtype="f16", page=0, mix=0),
        # A tree of 16 over one 32K conversation.
        dict(name="attend_32k_tree16", op="attend", B=1, L=32768, n=16, tree=True, Hq=32, Hkv=8, d=128,
             dtype="f16", page=0, mix=0),
        # A tree of 64 with eight heads per KV head: the matrix products count as much as the bytes.
        dict(name="attend_32k_tree64_g8", op="attend", B=1, L=32768, n=64, tree=True, Hq=64, Hkv=8,
             d=128, dtype="bf16", page=0, mix=0),
        # Ragged paged batch with sixteen heads per KV head: sequences without drafts or without a prefix.
        dict(name="attend_ragged_g16", op="attend", B=17, L=16384, n=9, tree=True, Hq=64, Hkv=4, d=128,
             dtype="bf16", page=64, mix=7),
        # A serving batch over an FP8 cache in small pages, chains of five.
        dict(name="attend_fp8_chain5", op="attend", B=64, L=4096, n=5, tree=False, Hq=32, Hkv=8, d=128,
             dtype="f16_e4m3kv", page=16, mix=0),
        # One 128K conversation over a 4-bit cache.
        dict(name="attend_4bit_128k", op="attend", B=1, L=131072, n=24, tree=True, Hq=64, Hkv=8, d=128,
             dtype="bf16_e2m1kv", page=0, mix=0),
        # The full serving batch: 64 conversations of 8K tokens, trees of 16.
        dict(name="attend_64x8k_tree16", op="attend", B=64, L=8192, n=16, tree=True, Hq=32, Hkv=8, d=128,
             dtype="bf16", page=0, mix=0),
        # The verdict on one tree: latency.
        dict(name="verify_one", op="verify", B=1, n=16, V=32768, tree=True, mix=0),
        # A serving batch of chains with the draft's probabilities.
        dict(name="verify_chains", op="verify", B=64, n=6, V=131072, tree=False, mix=0),
        # Ragged trees over a vocabulary of odd size.
        dict(name="verify_ragged", op="verify", B=17, n=33, V=50021, tree=True, mix=5),
        # The rows that stand, of one conversation: latency.
        dict(name="keep_one", op="keep", B=1, L=4097, n=16, Hq=32, Hkv=8, d=128, dtype="f16", page=64, mix=0),
        # The rows that stand, of a serving batch over an FP8 cache in small pages.
        dict(name="keep_64_fp8", op="keep", B=64, L=1024, n=64, Hq=32, Hkv=8, d=128, dtype="f16_e4m3kv",
             page=16, mix=3),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "attend", "verify", "verify", "keep"])
    c = dict(op=op, B=_log(rng, 1, 64), n=_log(rng, 1, 64), mix=rng.choice([0, rng.randrange(1, 1000)]))
    if op == "verify":
        c["tree"] = rng.random() < 0.5
        c["V"] = _log(rng, 1000, max(1001, min(131072, 50000000 // (c["B"] * c["n"]))))
        return c
    c["d"], c["Hkv"] = rng.choice([64, 128, 128]), rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 2, 3, 4, 5, 8, 16])
    c["Hq"] = G * c["Hkv"]
    c["page"] = rng.choice([0, 16, 32, 64, 128, 256])
    most = 400000 // (c["B"] * c["Hkv"])                  # tokens x KV heads of a drawn case stay below this
    if op == "attend":
        most = min(most, 200000000 // (c["B"] * c["Hq"] * c["n"]))
    c["L"] = max(c["n"], _log(rng, 1, max(1, min(40000, most))))
    if op == "attend":
        c["tree"] = rng.random() < 0.7
        c["dtype"] = rng.choice(["f16", "bf16", "f16_e4m3kv", "f16_e2m1kv", "bf16_e2m1kv"])
    else:
        c["dtype"] = rng.choice(["f16", "bf16", "f16_e4m3kv"])
    return c


# ------------------------------------------------------------------ shapes of a case

def _drafts(case):
    """Drafted tokens of each sequence: equal, or ragged, with sequences of none and of one."""
    B, n = case["B"], case["n"]
    if not case["mix"]:
        return [n] * B
    r = random.Random(case["mix"])
    some = [n, 0, 1][:B] + [r.randrange(1, n + 1) for _ in range(B - 3)]
    r.shuffle(some)
    return some


def _lengths(case):
    """Tokens of each sequence, the drafted ones included: equal, or ragged, one of them without a prefix."""
    some, L = _drafts(case), case.get("L", case["n"])
    if not case["mix"]:
        return [L] * case["B"]
    r = random.Random(case["mix"] + 1)
    return [max(n, L if b == 0 else 0 if b == 1 else _log(r, 1, L)) for b, n in enumerate(some)]


def _four(case):
    return "e2m1" in case["dtype"]


def _blocks(lens):
    """Rows of 16 tokens (4-bit) of a contiguous cache: every sequence starts a new one."""
    return [-(-x // 16) for x in lens]


def _row_bytes(case):
    """Bytes of one (token, KV head) of K or of V."""
    return case["d"] * 9 / 16 if _four(case) else case["d"] * (1 if "e4m3" in case["dtype"] else 2)


def work(case):
    some = _drafts(case)
    T, B = sum(some), case["B"]
    if case["op"] == "verify":
        # One row of the target for each sequence (and one of the draft), what the walk gathers, the answer.
        return {"bytes": max(1, sum(x > 0 for x in some) * 4 * case["V"] * (1 if case["tree"] else 2)
                             + T * 4 * 5 + B * (8 * max(some) + 4)), "flops": B * case["V"]}
    if case["op"] == "keep":
        row = case["Hkv"] * _row_bytes(case)
        moved = sum(max(0, _kept(x) - 1) for x in some)
        return {"bytes": max(1, 2 * 2 * moved * row + 4 * T), "flops": 0}
    # Sequences without drafted tokens are not read.
    N = sum(x for x, n in zip(_lengths(case), some) if n)
    pairs = sum(x * n for x, n in zip(_lengths(case), some))
    return {"bytes": max(1, N * 2 * case["Hkv"] * _row_bytes(case) + T * (case["Hq"] * (4 * case["d"] + 4) + 8)),
            "flops": 4 * pairs * case["Hq"] * case["d"]}


def _kept(n):
    """Rows that stand of n drafted ones: a third of them, the root among them."""
    return (n + 2) // 3


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

def _fill(case, pack, nrows, dev, gen, amp):
    """A cache of `nrows` rows (tokens, or blocks of 16 tokens) as earlier appends left it, its
    channels of sizes `amp`; `pack` lays out a 4-bit one."""
    H, d = case["Hkv"], case["d"]
    if not _four(case):
        x = torch.randn((nrows, H, d), device=dev, generator=gen)
        if "e4m3" in case["dtype"]:
            return (x * amp).to(torch.float8_e4m3fn).view(torch.uint8)
        return (x * amp).to(_Q[case["dtype"]])
    step = max(1, (1 << 25) // (16 * H * d))
    return torch.cat([pack(*_quantise(torch.randn((min(step, nrows - a), H, 16, d), device=dev, generator=gen) * amp))
                      for a in range(0, nrows, step)])


def _caches(s, gen, dev):
    """Caches (and page table) of the case, every sequence's last rows its drafted tokens."""
    case, lens = s["case"], s["lens"]
    page, d = case["page"], case["d"]
    unit = 16 if _four(case) else 1                       # tokens a cache row
    s["table"] = None
    if page:
        need = [-(-x // page) for x in lens]
        pages, most = sum(need) + 3, max(1, max(need))
        perm = torch.randperm(pages, device=dev, generator=gen).to(torch.int32)
        n = torch.tensor(need, device=dev)
        at = (torch.cumsum(n, 0) - n)[:, None] + torch.arange(most, device=dev)
        s["table"] = torch.where(torch.arange(most, device=dev) < n[:, None], perm[at.clamp(max=pages - 1)], 0).int()
        nrows = pages * page // unit
    else:
        n = torch.tensor([16 * x for x in _blocks(lens)] if _four(case) else lens, device=dev)
        s["first"] = torch.cumsum(n, 0) - n               # cache row of each sequence's first token
        nrows = max(1, int(n.sum()) // unit)
    # Keys have channels of different sizes; values do not.
    amp = torch.rand(d, device=dev, generator=gen) * 1.5 + 0.25
    pools = [_fill(case, _pack_k, nrows, dev, gen, amp), _fill(case, _pack_v, nrows, dev, gen, 1.0)]
    s["k_cache"], s["v_cache"] = [x.view(pages, page // unit, *x.shape[1:]) for x in pools] if page else pools


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    rng = random.Random(seed)
    some, lens = _drafts(case), _lengths(case)
    B, T, top = case["B"], sum(some), max(some)
    s = {"case": case, "some": some, "lens": lens, "kept": {}}     # kept: the plan, made at the first call
    n = torch.tensor(some, device=dev)
    s["n"] = n
    s["there"] = torch.arange(top, device=dev) < n[:, None]        # [B, most drafted]
    s["at"] = ((torch.cumsum(n, 0) - n)[:, None] + torch.arange(top, device=dev) * s["there"]).clamp(max=max(0, T - 1))
    # The trees: every token's parent among the eight before it, and the token with its ancestors as bits.
    parents, masks = [], []
    for m in some:
        up = [-1] + [rng.randrange(max(0, i - 8), i) for i in range(1, m)]
        bits = []
        for i in range(m):
            bits.append((1 << i) | (bits[up[i]] if i else 0))
        parents += up[:m]
        masks += [x - (1 << 64) if x >> 63 else x for x in bits]
    s["parents"] = s["mask"] = None
    if case.get("tree"):
        s["parents"] = torch.tensor(parents, dtype=torch.int32, device=dev)
        s["mask"] = torch.tensor(masks, dtype=torch.int64, device=dev)
    if case["op"] == "verify":
        V = case["V"]
        # Each row has three likely tokens among many unlikely ones.
        x = 4 * torch.randn((T, V), device=dev, generator=gen)
        x.scatter_(1, torch.randint(0, V, (T, 3), device=dev, generator=gen),
                   torch.tensor([20.0, 19.0, 18.0], device=dev).expand(T, 3))
        s["target"], s["draft"] = torch.softmax(x, -1), None
        if case["tree"]:
            # A drafting model's best tokens, in order: its first guess is often the target's.
            best = torch.topk(s["target"], 8).indices
            seen, pick, at = [0] * T, [], 0
            for m in some:
                for i in range(m):
                    up = at + max(0, parents[at + i])
                    pick.append((up, seen[up] % 8))
                    seen[up] += i > 0
                at += m
            pick = torch.tensor(pick, device=dev, dtype=torch.int64).view(T, 2)
            s["tokens"] = best[pick[:, 0], pick[:, 1]].int()
        else:
            # A token is drawn from what the draft says after the token before it.
            x = x.roll(1, 0) + 0.7 * torch.randn((T, V), device=dev, generator=gen)
            s["draft"] = torch.softmax(x, -1)
            s["tokens"] = torch.multinomial(s["draft"], 1, generator=gen)[:, 0].int() if T else \
                torch.zeros(0, dtype=torch.int32, device=dev)
        s["uniform"] = torch.rand(T, device=dev, generator=gen)
        return s
    _caches(s, gen, dev)
    if case["op"] == "attend":
        s["q"] = torch.randn((T, case["Hq"], case["d"]), device=dev, generator=gen).to(_Q[case["dtype"]])
        return s
    # What a verdict said: the root and ascending nodes below it.
    path = [[0] + sorted(rng.sample(range(1, m), _kept(m) - 1)) if m else [] for m in some]
    s["count"] = torch.tensor([len(p) for p in path], dtype=torch.int32, device=dev)
    s["path"] = torch.tensor([p + [-1] * (top - len(p)) for p in path], dtype=torch.int32, device=dev)
    return s


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


def _plain_attend(s):
    case, lens = s["case"], s["lens"]
    B, Hq, Hkv, d, top = case["B"], case["Hq"], case["Hkv"], case["d"], s["there"].shape[1]
    dev = s["q"].device
    most = max(lens)
    L = torch.tensor(lens, device=dev)[:, None]
    row = torch.arange(most, device=dev).expand(B, most)
    at = _pool_rows(s, torch.arange(B, device=dev)[:, None], row * (row < L))
    k, v = _cache_values(s)
    at = at.clamp(max=k.shape[0] - 1)                     # sequences without a token at the end
    k, v = k[at].transpose(1, 2), v[at].transpose(1, 2)   # [B, Hkv, most, d]
    node = row - (L - s["n"][:, None])                    # negative in the prefix
    if s["mask"] is not None:
        bit = (s["mask"][s["at"]][:, :, None] >> node.clamp(0, 63)[:, None]) & 1 == 1
    else:
        bit = node[:, None] <= torch.arange(top, device=dev)[None, :, None]
    sees = ((node < 0)[:, None] | bit) & (row < L)[:, None]        # [B, top, most]
    q = s["q"].float()[s["at"]]
    q = q.unflatten(2, (Hkv, Hq // Hkv)).permute(0, 2, 1, 3, 4).flatten(2, 3)    # [B, Hkv, top x group, d]
    x = (q @ k.mT).unflatten(2, (top, -1)) / math.sqrt(d)
    x = x.masked_fill(~sees[:, None, :, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = torch.exp(x - m)
    l = p.sum(-1, keepdim=True)
    out = (p.flatten(2, 3) @ v).unflatten(2, (top, -1))
    out = torch.where(l > 0, out / l, torch.zeros_like(out)).permute(0, 2, 1, 3, 4).reshape(B, top, Hq, d)
    lse = (m + torch.log(l))[..., 0].permute(0, 2, 1, 3).reshape(B, top, Hq)
    return {"out": out[s["there"]].to(_Q[case["dtype"]]), "lse": lse[s["there"]]}


def _plain_verify(s):
    there, at, V = s["there"], s["at"], s["target"].shape[1]
    B, top = there.shape
    i = torch.arange(top, device=at.device)
    up = s["parents"].long()[at] if s["parents"] is not None else (i - 1).expand(B, top)
    tok, u = s["tokens"].long()[at], s["uniform"].double()[at]
    child = there & (i > 0)
    p = torch.where(child, s["target"][at.gather(1, up.clamp(min=0)), tok].double(), 0.0)
    if s["draft"] is not None:
        stands = child & (u * s["draft"][at, tok].double() < p)
        sibling = torch.zeros((B, top, top), dtype=torch.bool, device=at.device)
    else:
        # sibling[i, j]: j is tried before i at the same node.
        sibling = (up[:, :, None] == up[:, None, :]) & (i[None, :] < i[:, None]) & child[:, :, None] & child[:, None, :]
        p = torch.where((sibling & (tok[:, :, None] == tok[:, None, :])).any(-1), 0.0, p)
        stands = child & (u * (1 - (sibling * p[:, None]).sum(-1)) < p)
    first = stands & ~(sibling & stands[:, None]).any(-1) | (i == 0) & there
    if s["mask"] is not None:
        above = (s["mask"][at][:, :, None] >> i) & 1 == 1
    else:
        above = (i[None, :] <= i[:, None]).expand(B, top, top)
    on = there & (first[:, None] | ~above).all(-1)
    count = on.sum(-1)
    path = torch.sort(torch.where(on, i, top)).values
    last = torch.where(on, i, 0).amax(-1)
    # The next token: from the last node's row, without the tokens tried there, or less their draft.
    w = s["target"][at.gather(1, last[:, None])[:, 0]].double()
    tried = child & (up == last[:, None])
    if s["draft"] is not None:
        left = (w - s["draft"][at.gather(1, (last + 1).clamp(max=top - 1)[:, None])[:, 0]].double()).clamp(min=0)
        left = torch.where(tried.any(-1, keepdim=True), left, w)
    else:
        gone = torch.zeros((B, V + 1), dtype=torch.bool, device=at.device)
        left = w.masked_fill(gone.scatter_(1, torch.where(tried, tok, V), True)[:, :V], 0.0)
    left = torch.where(left.sum(-1, keepdim=True) > 0, left, w)
    sums = torch.cumsum(left, -1)
    follow = torch.searchsorted(sums, u[:, :1] * sums[:, -1:], right=True)[:, 0].clamp(max=V - 1)
    said = tok.gather(1, path.roll(-1, 1).clamp(max=top - 1))
    said = torch.where(i == count[:, None] - 1, follow[:, None], said)
    past = i >= count[:, None]
    return {"path": path.masked_fill(past, -1).int(), "tokens": said.masked_fill(past, -1).int(), "count": count.int()}


def _plain_keep(s):
    case = s["case"]
    top = s["path"].shape[1]
    i = torch.arange(top, device=s["path"].device)
    stays = i < s["count"][:, None]
    sid = torch.arange(case["B"], device=i.device)[:, None].expand_as(stays)[stays]
    first = (torch.tensor(s["lens"], device=i.device) - s["n"])[sid]
    to = _pool_rows(s, sid, first + i.expand_as(stays)[stays])
    source = _pool_rows(s, sid, first + s["path"][stays].long())
    for name in ("k_cache", "v_cache"):
        pool = s[name].view(-1, case["Hkv"], case["d"])
        pool[to] = pool[source]
    return {"k_cache": _seen(s, "k_cache"), "v_cache": _seen(s, "v_cache")}


def _seen(s, name):
    """The whole cache as the numbers it holds."""
    return s[name].view(torch.float8_e4m3fn) if "e4m3" in s["case"]["dtype"] else s[name]


# ------------------------------------------------------------------ the framework's calls

def _tree(s):
    """The plan of a step's lengths and drafts (host memory) serves its attention in every layer."""
    if "tree" not in s["kept"]:
        import split_kv_flash_decode_gb300 as fd
        case = s["case"]
        s["kept"]["tree"] = fd.TreeDecoder(case.get("Hq", 32), case.get("Hkv", 8), case.get("d", 128), s["lens"],
                                           s["some"], case.get("dtype", "f16"), page_size=case.get("page", 0))
    return s["kept"]["tree"]


def _own(s):
    case, tree = s["case"], _tree(s)
    if case["op"] == "attend":
        out, lse = tree(s["q"], s["k_cache"], s["v_cache"], s["mask"], block_table=s["table"])
        return {"out": out, "lse": lse}
    if case["op"] == "verify":
        path, tokens, count = tree.verify(s["target"], s["tokens"], s["uniform"], parents=s["parents"],
                                          draft=s["draft"])
        return {"path": path, "tokens": tokens, "count": count}
    tree.keep(s["k_cache"], s["v_cache"], s["path"], s["count"], block_table=s["table"])
    return {"k_cache": _seen(s, "k_cache"), "v_cache": _seen(s, "v_cache")}


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    return _plain_attend(state) if op == "attend" else _plain_verify(state) if op == "verify" else _plain_keep(state)


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
    t = torch.arange(lo, hi, device="cuda")
    if s["table"] is None:
        per = [16 * x for x in _blocks(s["lens"])] if _four(case) else s["lens"]
        return t + sum(per[:b])
    return s["table"][b].long()[t // case["page"]] * case["page"] + t % case["page"]


def _exact_cache(s, name, rows):
    """Doubles of the given cache rows."""
    case, d, H = s["case"], s["case"]["d"], s["case"]["Hkv"]
    if _four(case):
        pool = s[name].view(-1, H, 9 * d)
        blocks, at = torch.unique(rows // 16, return_inverse=True)
        step = max(1, (1 << 24) // (16 * H * d))
        vals = [_exact_blocks(pool[blocks[i:i + step]], name[0], d) for i in range(0, blocks.numel(), step)]
        return torch.cat(vals)[at * 16 + rows % 16]
    t = torch.float8_e4m3fn if "e4m3" in case["dtype"] else _Q[case["dtype"]]
    return s[name].view(-1, H, d)[rows].view(t).double()


def exact(case, seed):
    s = prepare(case, seed)
    some, lens, B = s["some"], s["lens"], case["B"]
    first = [sum(some[:b]) for b in range(B)]
    if case["op"] == "verify":
        return _exact_verify(s, some, first)
    if case["op"] == "keep":
        done = []
        for name in ("k_cache", "v_cache"):
            t = torch.float8_e4m3fn if "e4m3" in case["dtype"] else _Q[case["dtype"]]
            pool = s[name].view(t).double()
            flat = pool.view(-1, case["Hkv"], case["d"])
            old = flat.clone()
            for b in range(B):
                rows = _exact_index(s, b, lens[b] - some[b], lens[b])
                for i, x in enumerate(s["path"][b, :int(s["count"][b])].tolist()):
                    flat[rows[i]] = old[rows[x]]
            done.append(pool)
        return {"k_cache": done[0], "v_cache": done[1]}
    Hq, Hkv, d = case["Hq"], case["Hkv"], case["d"]
    out = torch.zeros((sum(some), Hq, d), dtype=torch.float64, device="cuda")
    lse = torch.full((sum(some), Hq), -math.inf, dtype=torch.float64, device="cuda")
    bits = s["mask"].tolist() if s["mask"] is not None else None
    for b in range(B):
        n, L = some[b], lens[b]
        if n == 0:
            continue
        rows = _exact_index(s, b, 0, L)
        k, v = _exact_cache(s, "k_cache", rows), _exact_cache(s, "v_cache", rows)
        hide = torch.zeros((n, L), dtype=torch.bool)
        for i in range(n):
            for j in range(n):
                hide[i, L - n + j] = j > i if bits is None else not bits[first[b] + i] >> j & 1
        hide = hide.cuda()
        q = s["q"][first[b]:first[b] + n].double().view(n, Hkv, Hq // Hkv, d)
        for h in range(Hkv):
            x = torch.einsum("ngd,ld->ngl", q[:, h], k[:, h]) / d ** 0.5
            x = x.masked_fill(hide[:, None], -math.inf)
            at = slice(h * (Hq // Hkv), (h + 1) * (Hq // Hkv))
            lse[first[b]:first[b] + n, at] = torch.logsumexp(x, -1)
            out[first[b]:first[b] + n, at] = torch.einsum("ngl,ld->ngd", torch.softmax(x, -1), v[:, h])
    return {"out": out, "lse": lse}


def _exact_verify(s, some, first):
    """The walk itself, node by node, on the host."""
    top = max(some)
    path = torch.full((len(some), top), -1, dtype=torch.int32)
    said, count = path.clone(), torch.zeros(len(some), dtype=torch.int32)
    u, tok = s["uniform"].double().tolist(), s["tokens"].tolist()
    up = s["parents"].tolist() if s["parents"] is not None else None
    for b, n in enumerate(some):
        a, node, got, words = first[b], 0, [0], []
        if n == 0:
            continue
        while True:
            below = [i for i in range(1, n) if (up[a + i] if up else i - 1) == node]
            row = s["target"][a + node].double()
            left, mass, went = row.clone(), 1.0, None
            for i in below:
                x = tok[a + i]
                if s["draft"] is not None:
                    other = s["draft"][a + i].double()
                    if u[a + i] * float(other[x]) < float(row[x]):
                        went = i
                        break
                    left = torch.relu(row - other)
                else:
                    if u[a + i] * mass < float(left[x]):
                        went = i
                        break
                    mass -= float(left[x])
                    left[x] = 0.0
            if went is None:
                break
            node = went
            got.append(node)
            words.append(tok[a + node])
        sums = torch.cumsum(left if float(left.sum()) > 0 else row, 0)
        words.append(min(int((sums <= u[a] * sums[-1]).sum()), sums.numel() - 1))
        path[b, :len(got)] = torch.tensor(got, dtype=torch.int32)
        said[b, :len(got)] = torch.tensor(words, dtype=torch.int32)
        count[b] = len(got)
    return {"path": path, "tokens": said, "count": count}
