"""What the attention beside the indexer costs: workloads of the operators that read, fill and thin out
the caches whose tokens the indexer selects.

Four operators, each with its plain form (elementary torch operations in fp32) and its call into the
library:

  cache    misa_kv4_append + misa_kv4_read: keys and values written to a paged cache in 4 bits and read back
  decode   misa_kv4_attention: one query token per sequence over that cache, over the whole prefix or over
           the tokens the indexer selected, adding each token's attention weight to a running sum if asked
  evict    misa_evict_select + misa_kv4_compact + misa_keys_compact_paged: the tokens with the largest
           summed weight stay, and the caches close up in place
  prompt   misa_prompt_attention: causal attention of packed prompts with grouped heads, or of the last
           queries of a longer sequence

The cache holds e2m1 codes (0, 0.5, 1, 1.5, 2, 3, 4, 6 with a sign) with one e4m3 scale per 16 elements.  A
pool is uint8 [pages, kv heads, 2 (K, V), page_size * 9 d / 16]; such a slab holds page_size code rows of d/2
bytes, then page_size scale rows of d/16 bytes.  Code row: byte (d/8) c + 2 j + i holds elements
16 j + 4 c + 2 i (low nibble) and the next one (high nibble), for c < 4, j < d/16, i < 2.
"""
import math
import random

import torch

own = False

LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    return [
        # a few short chat turns answered together: every length ragged, one a single token (latency)
        dict(name="prompt_short", op="prompt", S=4, lo=1, hi=300, prefix=0, Hq=8, Hkv=2, d=64, mix=1),
        # an ordinary prefill batch of packed prompts of different lengths, grouped heads 4:1
        dict(name="prompt_packed", op="prompt", S=12, lo=200, hi=4096, prefix=0, Hq=32, Hkv=8, d=128, mix=2),
        # chunked prefill: 4096 queries that end a 32K prompt
        dict(name="prompt_chunk", op="prompt", S=1, lo=4096, hi=4096, prefix=28672, Hq=16, Hkv=2, d=128, mix=3),
        # packed prompts entering the 4-bit cache, read back for the next chunk
        dict(name="cache_prompt", op="cache", S=3, lo=2000, hi=9000, prefix=37, Hkv=8, d=128, page=64, mix=4),
        # one new token for each of 32 decoding sequences
        dict(name="cache_token", op="cache", S=32, lo=1, hi=1, prefix=1000, Hkv=8, d=128, page=64, mix=5),
        # a single conversation's token: the smallest call, where latency counts
        dict(name="decode_one", op="decode", T=1, lo=1000, hi=1000, Hq=32, Hkv=8, d=128, page=64, pick=0, acc=False, f32=False, mix=6),
        # a serving batch of ragged prefixes whose attention weights are summed for eviction
        dict(name="decode_batch", op="decode", T=32, lo=500, hi=16384, Hq=32, Hkv=8, d=128, page=64, pick=0, acc=True, f32=False, mix=7),
        # sixteen sequences at full context
        dict(name="decode_long", op="decode", T=16, lo=120000, hi=131072, Hq=64, Hkv=8, d=128, page=64, pick=0, acc=False, f32=False, mix=8),
        # fp32 queries, 64-wide heads, groups of 3, small pages, one prefix empty
        dict(name="decode_f32", op="decode", T=9, lo=0, hi=5000, Hq=12, Hkv=4, d=64, page=16, pick=0, acc=False, f32=True, mix=9),
        # the tokens the indexer picked (top 2048) of 32 sequences, their weights summed
        dict(name="decode_picked", op="decode", T=32, lo=1500, hi=32768, Hq=64, Hkv=8, d=128, page=64, pick=2048, acc=True, f32=False, mix=10),
        # a batch of long caches thinned to a quarter of the largest
        dict(name="evict_batch", op="evict", T=16, lo=4000, hi=32768, keep=8192, sink=4, recent=512, Hkv=8, d=128, page=64, mix=11),
        # one sequence over its small budget
        dict(name="evict_one", op="evict", T=1, lo=1000, hi=1000, keep=512, sink=4, recent=64, Hkv=4, d=64, page=16, mix=12),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op, mix = rng.choice(("prompt", "cache", "decode", "decode", "evict")), rng.randrange(1 << 20)
    d, Hkv = rng.choice((64, 128, 128)), _log(rng, 1, 8)
    page = rng.choice((16, 32, 64, 128))
    if op == "prompt":
        S, G = _log(rng, 1, 12), _log(rng, 1, 32 // Hkv)
        hi, prefix = _log(rng, 16, 4096), rng.choice((0, 0, _log(rng, 1, 28672)))
        S = max(1, min(S, int(3e9 / (G * Hkv * hi * (hi + prefix)))))
        return dict(op=op, S=S, lo=_log(rng, 1, hi), hi=hi, prefix=prefix, Hq=Hkv * G, Hkv=Hkv, d=d, mix=mix)
    if op == "cache":
        S = _log(rng, 1, 32)
        hi = _log(rng, 1, 24000 // S)
        return dict(op=op, S=S, lo=_log(rng, 1, hi), hi=hi, prefix=_log(rng, 1, 1000), Hkv=Hkv, d=d, page=page, mix=mix)
    T, hi = _log(rng, 1, 32), _log(rng, 8, 131072 if op == "decode" else 32768)
    lo = _log(rng, 1, hi)
    if op == "decode":
        T = max(1, min(T, (1 << 23) // (hi * Hkv)))
        pick = rng.choice((0, 0, _log(rng, 1, 2048)))
        return dict(op=op, T=T, lo=rng.choice((0, lo)), hi=hi, Hq=Hkv * _log(rng, 1, 16), Hkv=Hkv, d=d, page=page, pick=pick,
                    acc=rng.random() < 0.5, f32=rng.random() < 0.25, mix=mix)
    keep = _log(rng, 4, max(5, hi // 2))
    return dict(op=op, T=min(T, 16), lo=lo, hi=hi, keep=keep, sink=min(4, keep // 4), recent=keep // 8, Hkv=Hkv, d=d, page=page, mix=mix)


def _lengths(case, count):
    """Lengths from lo to hi, spread over their logarithm, the largest among them (and lo, where there are two or more)."""
    r, lo, hi = random.Random(case["mix"]), case["lo"], case["hi"]
    got = [_log(r, max(1, lo), max(1, hi)) for _ in range(count)]
    got[0] = hi
    if count > 1:
        got[-1] = lo
    return got


def _cumulative(lengths):
    got = [0]
    for x in lengths:
        got.append(got[-1] + x)
    return got


def _tables(g, count, tokens, page):
    """Page tables [count, pages] over a shuffled pool that has a few pages more."""
    per = -(-tokens // page)
    total = count * per + 3
    return torch.randperm(total, generator=g, device="cuda")[: count * per].to(torch.int32).view(count, per), total


def _random_pool(g, total, Hkv, page, d):
    """A pool as appends leave it: any code, scales of blocks whose largest element lies between 0.4 and 3."""
    pool = torch.randint(0, 256, (total, Hkv, 2, page * 9 * d // 16), generator=g, device="cuda", dtype=torch.uint8)
    scales = pool[..., page * d // 2:]
    scales.copy_((scales & 15) + 0x18)
    return pool


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    f = dict(generator=g, device="cuda")
    st = dict(case)
    i32 = dict(dtype=torch.int32, device="cuda")
    op = case["op"]
    if op == "prompt":
        lens = _lengths(case, case["S"])
        cu_q, cu_k = _cumulative(lens), _cumulative([x + case["prefix"] for x in lens])
        st["lens"] = lens
        st["q"] = torch.randn(cu_q[-1], case["Hq"], case["d"], **f).mul_(1.5).bfloat16()
        st["k"] = torch.randn(cu_k[-1], case["Hkv"], case["d"], **f).bfloat16()
        st["v"] = torch.randn(cu_k[-1], case["Hkv"], case["d"], **f).bfloat16()
        st["cu_q"], st["cu_k"] = torch.tensor(cu_q, **i32), torch.tensor(cu_k, **i32)
    elif op == "cache":
        lens = _lengths(case, case["S"])
        cu = _cumulative(lens)
        st["cu"], st["start"] = torch.tensor(cu, **i32), torch.full((case["S"],), case["prefix"], **i32)
        st["table"], total = _tables(g, case["S"], case["prefix"] + max(lens), case["page"])
        st["pool"] = _random_pool(g, total, case["Hkv"], case["page"], case["d"])
        shape = (cu[-1], case["Hkv"], case["d"])
        st["k"] = torch.randn(shape, **f).mul_(torch.rand(case["d"], **f).mul_(3).add_(0.3)).bfloat16()
        st["v"] = torch.randn(shape, **f).mul_(0.05).bfloat16()
        st["k_scale"], st["v_scale"] = 1.0, 2.0 ** -5
    elif op == "decode":
        T, lens = case["T"], _lengths(case, case["T"])
        L = max(lens)
        st["n"] = torch.tensor(lens, **i32)
        st["table"], total = _tables(g, T, L, case["page"])
        st["pool"] = _random_pool(g, total, case["Hkv"], case["page"], case["d"])
        st["q"] = torch.randn(T, case["Hq"], case["d"], **f).to(torch.float32 if case["f32"] else torch.bfloat16)
        st["idx"] = None
        if case["pick"]:  # distinct tokens of the prefix in no order, -1 behind them
            key = torch.rand(T, L, **f).masked_fill_(torch.arange(L, device="cuda")[None] >= st["n"][:, None], 2.0)
            val, at = key.sort(dim=1)
            at = torch.where(val > 1.5, -1, at).to(torch.int32)[:, : case["pick"]]
            st["idx"] = torch.nn.functional.pad(at, (0, case["pick"] - at.shape[1]), value=-1).contiguous()
        st["acc"] = torch.rand(T, L, **f) if case["acc"] else None
    else:
        T, lens = case["T"], _lengths(case, case["T"])
        L = max(lens)
        st["n"] = torch.tensor(lens, **i32)
        st["table"], total = _tables(g, T, L, case["page"])
        st["pool"] = _random_pool(g, total, case["Hkv"], case["page"], case["d"])
        st["keys"] = torch.randn(total, case["page"], 128, **f).bfloat16()
        # summed weights fall off as a power; the smallest are cut to zero, so that there are ties
        acc = torch.rand(T, L, **f).add_(1e-3).pow_(-0.7).sub_(1.1).clamp_(min=0.0)
        st["acc"] = acc
    return st


# ---- plain forms ----------------------------------------------------------------------------------------------------


def _levels(device, dtype=torch.float32):
    """[256, 2]: what the low and the high nibble of a byte stand for."""
    one = torch.tensor(LEVELS, dtype=dtype, device=device)
    both = torch.cat([one, -one])
    b = torch.arange(256, device=device)
    return torch.stack([both[b & 15], both[b >> 4]], dim=1)


def _unpack(codes, scales, dtype=torch.float32):
    """codes uint8 [..., d/2], scales uint8 [..., d/16] -> values [..., d]."""
    lead, nb = codes.shape[:-1], scales.shape[-1]
    x = _levels(codes.device, dtype).index_select(0, codes.reshape(-1).to(torch.int32)).view(*lead, 4, nb, 2, 2)
    x = x.movedim(-4, -3).reshape(*lead, nb, 16)
    s = scales.contiguous().view(torch.float8_e4m3fn).to(dtype)
    return (x * s.unsqueeze(-1)).view(*lead, nb * 16)


def _pack(x, scale):
    """x [..., d] -> codes, scales: s = e4m3(max|x| / (6 scale)) per 16 elements, each x / (s scale) to the nearest level, ties to the even code."""
    lead, nb = x.shape[:-1], x.shape[-1] // 16
    x = x.float().view(*lead, nb, 16)
    g = torch.full((1,), scale, dtype=torch.float32, device=x.device)
    s8 = (x.abs().amax(-1) / (g * 6.0)).clamp(max=448.0).to(torch.float8_e4m3fn)
    y = x / (s8.float() * g).unsqueeze(-1)
    m = y.abs()
    c = (m > 0.25).to(torch.uint8) + (m >= 0.75) + (m > 1.25) + (m >= 1.75) + (m > 2.5) + (m >= 3.5) + (m > 5.0)
    c = c + torch.signbit(y).to(torch.uint8) * 8
    c = torch.where(s8.float().unsqueeze(-1) == 0, torch.zeros_like(c), c)
    c = c.view(*lead, nb, 4, 2, 2).movedim(-4, -3)
    return (c[..., 0] | (c[..., 1] << 4)).reshape(*lead, nb * 8), s8.view(torch.uint8)


def _parts(pool, page, d):
    """Code rows [pages, Hkv, 2, page, d/2] and scale rows [pages, Hkv, 2, page, d/16] of a pool, as views."""
    a, b = pool[..., : page * d // 2], pool[..., page * d // 2:]
    return a.unflatten(-1, (page, d // 2)), b.unflatten(-1, (page, d // 16))


def _place(table, seq, pos, page):
    """Physical page and slot of logical positions pos of sequences seq."""
    return table[seq, pos // page].long(), pos % page


def _rows_of(cu, start, rows):
    r = torch.arange(rows, device=cu.device)
    seq = torch.searchsorted(cu[1:].long(), r, right=True)
    return seq, r - cu[seq] + start[seq]


def _cache_plain(st):
    page, d = st["page"], st["d"]
    codes, scales = _parts(st["pool"], page, d)
    seq, pos = _rows_of(st["cu"], st["start"], st["k"].shape[0])
    pg, at = _place(st["table"], seq, pos, page)
    for side, (x, scale) in enumerate(((st["k"], st["k_scale"]), (st["v"], st["v_scale"]))):
        codes[pg, :, side, at], scales[pg, :, side, at] = _pack(x, scale)
    back = [(_unpack(codes[pg, :, side, at], scales[pg, :, side, at]) * scale).bfloat16()
            for side, scale in ((0, st["k_scale"]), (1, st["v_scale"]))]
    return {"k": back[0], "v": back[1]}


def _soft(s, empty):
    """Softmax weights of s (in place) and its log of the sum of exps, over the last axis; a row with nothing to attend weighs nothing."""
    top = s.amax(-1, keepdim=True).masked_fill_(empty, 0.0)
    total = s.sub_(top).exp_().sum(-1, keepdim=True)
    s.div_(total.masked_fill(empty, 1.0))
    return s, (top + total.log()).squeeze(-1)


def _decode_plain(st):
    T, Hq, Hkv, d, page = st["T"], st["Hq"], st["Hkv"], st["d"], st["page"]
    n = st["n"].long()
    codes, scales = _parts(st["pool"], page, d)
    if st["idx"] is None:
        pos = torch.arange(int(st["hi"]), device="cuda").expand(T, -1)
        seen = pos < n[:, None]
    else:
        pos = st["idx"].long()
        seen = pos >= 0
        pos = pos.clamp(min=0)
    pg, at = _place(st["table"], torch.arange(T, device="cuda")[:, None], pos, page)
    q = st["q"].float().view(T, Hkv, Hq // Hkv, d) / math.sqrt(d)
    k = _unpack(codes[pg, :, 0, at], scales[pg, :, 0, at])  # [T, P, Hkv, d]
    s = q @ k.permute(0, 2, 3, 1)
    del k
    s = s.masked_fill_(~seen[:, None, None, :], -math.inf)
    p, lse = _soft(s, ~seen.any(-1)[:, None, None, None])
    v = _unpack(codes[pg, :, 1, at], scales[pg, :, 1, at])
    out = {"out": (p @ v.transpose(1, 2)).reshape(T, Hq, d).to(st["q"].dtype), "lse": lse.reshape(T, Hq)}
    if st["acc"] is not None:
        out["acc"] = st["acc"].scatter_add_(1, pos, p.sum((1, 2)))
    return out


def _evict_plain(st):
    T, keep, sink, recent, page = st["T"], st["keep"], st["sink"], st["recent"], st["page"]
    acc, n = st["acc"], st["n"].long()[:, None]
    L = acc.shape[1]
    s = torch.arange(L, device="cuda").expand(T, -1)
    held = (s < sink) | (s >= n - recent)
    order = acc.masked_fill(held | (s >= n), -1.0).sort(dim=1, descending=True, stable=True).indices
    rank = torch.empty_like(order).scatter_(1, order, s.contiguous())
    stay = (s < n) & ((n <= keep) | held | (rank < keep - sink - recent))
    idx = torch.where(stay, s, L).sort(dim=1).values[:, :keep]
    idx = torch.nn.functional.pad(idx, (0, keep - idx.shape[1]), value=L)
    live = idx < L
    new = torch.where(live, acc.gather(1, idx.clamp(max=L - 1)), 0.0)
    codes, scales = _parts(st["pool"], page, st["d"])
    j = torch.arange(idx.shape[1], device="cuda").clamp(max=L - 1).expand(T, -1)
    seq = torch.arange(T, device="cuda")[:, None]
    src, dst = _place(st["table"], seq, torch.where(live, idx, j), page), _place(st["table"], seq, j, page)
    for x in (codes, scales):
        x[dst[0], :, :, dst[1]] = x[src[0], :, :, src[1]]
    st["keys"][dst] = st["keys"][src]
    return {"idx": torch.where(live, idx, -1).to(torch.int32), "n": live.sum(1).to(torch.int32), "acc": new,
            "pool": st["pool"], "keys": st["keys"]}


def _padded(x, lens):
    """Packed rows [sum(lens), H, d] as [S, max(lens), H, d] fp32, and which rows are there."""
    at = torch.tensor(_cumulative(lens)[:-1], device=x.device)
    r = torch.arange(max(lens), device=x.device)
    there = r[None] < torch.tensor(lens, device=x.device)[:, None]
    return x[torch.where(there, at[:, None] + r, 0)].float() * there[..., None, None], there


def _prompt_plain(st):
    Hq, Hkv, d, lens = st["Hq"], st["Hkv"], st["d"], st["lens"]
    klens = [x + st["prefix"] for x in lens]
    q, there = _padded(st["q"], lens)
    k, kthere = _padded(st["k"], klens)
    v, _ = _padded(st["v"], klens)
    S, Lq, Lk = len(lens), max(lens), max(klens)
    q = q.view(S, Lq, Hkv, Hq // Hkv, d).permute(0, 2, 3, 1, 4) / math.sqrt(d)
    s = q @ k.permute(0, 2, 3, 1).unsqueeze(2)  # [S, Hkv, G, Lq, Lk]
    row, col = torch.arange(Lq, device="cuda")[:, None], torch.arange(Lk, device="cuda")
    hidden = (col > row + st["prefix"]) | ~kthere[:, None, None, None, :]
    s.masked_fill_(hidden, -math.inf)
    p, lse = _soft(s, hidden.all(-1, keepdim=True))
    o = (p @ v.transpose(1, 2).unsqueeze(2)).permute(0, 3, 1, 2, 4).reshape(S, Lq, Hq, d)
    return {"out": o[there].bfloat16(), "lse": lse.permute(0, 3, 1, 2).reshape(S, Lq, Hq)[there]}


# ---- the library's calls --------------------------------------------------------------------------------------------


def _own(st):
    from long_context_sparse_mean_b200 import binding as M

    op = st["op"]
    if op == "prompt":
        out, lse = M.misa_prompt_attention(st["q"], st["k"], st["v"], st["cu_q"], st["cu_k"], want_lse=True)
        return {"out": out, "lse": lse}
    if op == "cache":
        a = dict(k_scale=st["k_scale"], v_scale=st["v_scale"])
        M.misa_kv4_append(st["k"], st["v"], st["pool"], st["table"], st["cu"], st["start"], **a)
        k, v = M.misa_kv4_read(st["pool"], st["table"], st["cu"], st["start"], st["k"].shape[0], st["d"], **a)
        return {"k": k, "v": v}
    if op == "decode":
        out, lse = M.misa_kv4_attention(st["q"], st["pool"], st["table"], st["n"], idx=st["idx"], acc=st["acc"], want_lse=True)
        got = {"out": out, "lse": lse}
        if st["acc"] is not None:
            got["acc"] = st["acc"]
        return got
    idx, n, acc = M.misa_evict_select(st["acc"], st["n"], st["keep"], sink=st["sink"], recent=st["recent"], want_acc=True)
    M.misa_kv4_compact(st["pool"], st["table"], idx, st["d"])
    M.misa_keys_compact_paged(st["keys"], st["table"], idx)
    return {"idx": idx, "n": n, "acc": acc, "pool": st["pool"], "keys": st["keys"]}


def run(state):
    if own:
        return _own(state)
    plain = {"prompt": _prompt_plain, "cache": _cache_plain, "decode": _decode_plain, "evict": _evict_plain}
    return plain[state["op"]](state)


# ---- what a pass cannot do without ----------------------------------------------------------------------------------


def work(case):
    op, Hkv, d = case["op"], case["Hkv"], case["d"]
    row = Hkv * 2 * (d // 2 + d // 16)  # a token's K and V in the cache
    if op == "prompt":
        lens, pre, Hq = _lengths(case, case["S"]), case["prefix"], case["Hq"]
        rows = sum(lens)
        pairs = sum(x * pre + x * (x + 1) // 2 for x in lens)
        return {"bytes": rows * Hq * d * 4 + rows * Hq * 4 + (rows + pre * len(lens)) * Hkv * d * 4, "flops": 4 * d * Hq * pairs}
    if op == "cache":
        rows = sum(_lengths(case, case["S"]))
        return {"bytes": 2 * rows * (Hkv * d * 4 + row), "flops": 2 * rows * Hkv * d * 4}
    if op == "decode":
        lens, Hq = _lengths(case, case["T"]), case["Hq"]
        seen = sum(min(x, case["pick"]) if case["pick"] else x for x in lens)
        b = seen * row + case["T"] * Hq * (d * (8 if case["f32"] else 4) + 4)
        b += seen * 8 * case["acc"] + case["T"] * case["pick"] * 4
        return {"bytes": b, "flops": 4 * seen * Hq * d}
    lens = _lengths(case, case["T"])
    kept = sum(min(x, case["keep"]) for x in lens)
    moved = sum(case["keep"] for x in lens if x > case["keep"])
    return {"bytes": sum(lens) * 4 + case["T"] * case["keep"] * 8 + kept * 4 + 2 * moved * (row + 256), "flops": sum(lens)}


# ---- the definitions in 64 bits -------------------------------------------------------------------------------------


def _value64(codes, scales):
    """Rows of codes and scales as doubles, element by element of the row's layout."""
    d = codes.shape[-1] * 2
    e = torch.arange(d, device=codes.device)
    byte = (d // 8) * (e % 16 // 4) + 2 * (e // 16) + e % 4 // 2
    nib = (codes[..., byte].int() >> (4 * (e % 2)).int()) & 15
    ex, man = (nib >> 1) & 3, (nib & 1).double()
    mag = torch.where(ex == 0, man * 0.5, torch.exp2((ex - 1).double()) * (1.0 + man * 0.5))
    sb = scales[..., e // 16].int()
    sx, sm = (sb >> 3) & 15, (sb & 7).double() / 8
    scale = torch.where(sx == 0, sm * 2.0 ** -6, torch.exp2((sx - 7).double()) * (1.0 + sm))
    return torch.where(nib >= 8, -mag, mag) * scale


def _attend64(q, k, v, hidden=None):
    """q [H, m, d], k and v [H, l, d] doubles: the formula, with the rows that see nothing zero and minus infinity."""
    s = torch.einsum("hmd,hld->hml", q, k) / math.sqrt(q.shape[-1])
    if hidden is not None:
        s = s.masked_fill(hidden, -math.inf)
    lse = torch.logsumexp(s, dim=-1)
    p = torch.exp(s - torch.where(torch.isfinite(lse), lse, 0.0)[..., None])
    return torch.einsum("hml,hld->hmd", p, v), lse, p


def exact(case, seed):
    st = prepare(case, seed)
    op, Hkv, d = case["op"], case["Hkv"], case["d"]
    if op == "prompt":
        Hq, G, pre = case["Hq"], case["Hq"] // case["Hkv"], case["prefix"]
        outs, lses, at = [], [], 0
        for b, m in enumerate(st["lens"]):
            kat = at + b * pre
            o, z = torch.empty(m, Hq, d, dtype=torch.float64, device="cuda"), torch.empty(m, Hq, dtype=torch.float64, device="cuda")
            for h in range(Hq):
                k, v = (x[kat: kat + pre + m, h // G].double()[None] for x in (st["k"], st["v"]))
                for r in range(0, m, 2048):
                    e = min(m, r + 2048)
                    hide = torch.arange(pre + e, device="cuda")[None] > torch.arange(r, e, device="cuda")[:, None] + pre
                    got = _attend64(st["q"][at + r: at + e, h].double()[None], k[:, : pre + e], v[:, : pre + e], hide)
                    o[r:e, h], z[r:e, h] = got[0][0], got[1][0]
            outs.append(o)
            lses.append(z)
            at += m
        return {"out": torch.cat(outs), "lse": torch.cat(lses)}
    if op == "cache":
        got = {}
        grid = torch.tensor(LEVELS, dtype=torch.float64, device="cuda")
        for name in ("k", "v"):
            g = st[name + "_scale"]
            x = st[name].double().unflatten(-1, (d // 16, 16))
            raw = x.abs().amax(-1) / (6 * g)
            step = torch.exp2(torch.floor(torch.log2(raw.clamp(min=2.0 ** -6))) - 3)  # e4m3: 3 bits of fraction, steps of 2^-9 at least
            s = (torch.round(raw / step) * step).clamp(max=448.0)
            unit = (s * g).unsqueeze(-1)
            y = torch.where(unit > 0, x.abs() / unit.clamp(min=1e-300), 0.0)
            hi = torch.bucketize(y, grid).clamp(max=7)
            lo = (hi - 1).clamp(min=0)
            up = (y - grid[lo] > grid[hi] - y) | ((y - grid[lo] == grid[hi] - y) & (hi % 2 == 0))
            got[name] = (torch.copysign(torch.where(up, grid[hi], grid[lo]) * unit, x)).flatten(-2)
        return got
    T, lens = case["T"], _lengths(case, case["T"])
    if op == "decode":
        G, page = case["Hq"] // Hkv, case["page"]
        if sum(lens) * Hkv * d > 3e9:
            return None
        codes, scales = _parts(st["pool"], page, d)
        out = torch.zeros(T, case["Hq"], d, dtype=torch.float64, device="cuda")
        lse = torch.full((T, case["Hq"]), -math.inf, dtype=torch.float64, device="cuda")
        acc = st["acc"].double() if case["acc"] else None
        for t, n in enumerate(lens):
            pos = torch.arange(n, device="cuda") if st["idx"] is None else st["idx"][t][st["idx"][t] >= 0].long()
            if not len(pos):
                continue
            pg, at = st["table"][t].long()[pos // page], pos % page
            for h in range(Hkv):
                k, v = (_value64(codes[pg, h, side, at], scales[pg, h, side, at])[None] for side in (0, 1))
                o, z, p = _attend64(st["q"][t, h * G: (h + 1) * G].double()[None], k, v)
                out[t, h * G: (h + 1) * G], lse[t, h * G: (h + 1) * G] = o[0], z[0]
                if acc is not None:
                    acc[t, pos] += p[0].sum(0)
        return {"out": out, "lse": lse, **({"acc": acc} if case["acc"] else {})}
    keep, sink, recent, page = case["keep"], case["sink"], case["recent"], case["page"]
    keys = st["keys"].double()
    acc = torch.zeros(T, keep, dtype=torch.float64, device="cuda")
    for t, n in enumerate(lens):
        a = st["acc"][t, :n].double().cpu().tolist()
        if n > keep:
            mid = sorted(range(sink, n - recent), key=lambda s: (-a[s], s))[: keep - sink - recent]
            stay = sorted(list(range(sink)) + mid + list(range(n - recent, n)))
        else:
            stay = list(range(n))
        pos = torch.tensor(stay, dtype=torch.long, device="cuda")
        acc[t, : len(stay)] = st["acc"][t, pos].double()
        j, table = torch.arange(len(stay), device="cuda"), st["table"][t].long()
        keys[table[j // page], j % page] = keys[table[pos // page], pos % page]
    return {"idx": None, "n": None, "acc": acc, "pool": None, "keys": keys}
