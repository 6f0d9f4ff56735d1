"""The calls of a serving loop together: a prompt is attended to and written to the 4-bit cache, decode steps
select tokens with the indexer and attend to them, the caches are thinned by the weights they gathered, and
decoding goes on over what is left."""
import numpy as np
import pytest
import torch

import attention_ref as R
from gpu_common import host, lib

pytestmark = pytest.mark.gpu


def cuda(x, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(x)).cuda()
    return t if dtype is None else t.to(dtype)


def test_prompt_decode_evict_decode():
    M = lib()
    rng = np.random.default_rng(21)
    T, Hq, Hkv, d, page, H_I, B, h, topk = 3, 16, 2, 128, 64, 16, 32, 4, 64
    lens = [700, 233, 512]
    per = -(-(max(lens) + 8) // page)
    total = T * per
    table_h = rng.permutation(total).reshape(T, per).astype(np.int32)
    table = cuda(table_h)
    pool, keys = M.misa_kv4_pool(total, page, Hkv, d), torch.zeros(total, page, 128, dtype=torch.bfloat16, device="cuda")
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    rows = int(cu[-1])
    randn = lambda *s: cuda(rng.standard_normal(s).astype(np.float32), torch.bfloat16)  # noqa: E731
    q, k, v, ik = randn(rows, Hq, d), randn(rows, Hkv, d), randn(rows, Hkv, d), randn(rows, 128)

    # the prompt: attention in bf16, then the cache; the second half of it as a chunk over what was cached
    out, _ = M.misa_prompt_attention(q, k, v, cuda(cu))
    zero = cuda(np.zeros(T, np.int32))
    M.misa_kv4_append(k, v, pool, table, cuda(cu), zero)
    kb, vb = M.misa_kv4_read(pool, table, cuda(cu), zero, rows, d)
    half = [n // 2 for n in lens]
    cu_h = np.concatenate([[0], np.cumsum([n - a for n, a in zip(lens, half)])]).astype(np.int32)
    qh = torch.cat([q[cu[b] + half[b]:cu[b + 1]] for b in range(T)])
    chunk, _ = M.misa_prompt_attention(qh, kb, vb, cuda(cu_h), cuda(cu))
    for b in range(T):
        m, n = lens[b] - half[b], lens[b]
        seen = np.arange(n)[None] <= (np.arange(m) + n - m)[:, None]
        kk, vv, qq = (host(x.float()) for x in (kb[cu[b]:cu[b + 1]], vb[cu[b]:cu[b + 1]], qh[cu_h[b]:cu_h[b + 1]]))
        want, _, p = R.attend(qq, kk, vv, d ** -0.5, seen)
        tol, _ = R.attend_tolerance(qq, kk, vv, d ** -0.5, p, "bf16", 2.0 ** -8)
        assert np.all(np.abs(host(chunk[cu_h[b]:cu_h[b + 1]].float()) - want) <= tol)
        pos = torch.arange(lens[b], device="cuda")
        keys[table[b].long()[pos // page], pos % page] = ik[cu[b]:cu[b + 1]]

    n = cuda(np.array(lens, np.int32))
    acc = torch.zeros(T, per * page, device="cuda")
    acc_ref = np.zeros((T, per * page))
    nh = np.array(lens)

    def step():
        """One decode step of every sequence; checks attention against the cache's own values."""
        nonlocal nh
        one, k1, v1, ik1 = randn(T, Hq, d), randn(T, Hkv, d), randn(T, Hkv, d), randn(T, 128)
        M.misa_kv4_append(k1, v1, pool, table, cuda(np.arange(T + 1, dtype=np.int32)), n)
        for t in range(T):
            keys[table_h[t, nh[t] // page], nh[t] % page] = ik1[t]
        n.add_(1)
        nh = nh + 1
        kbar = M.misa_pool_keys_paged(keys, table, B)
        iq, iw = randn(T, H_I, 128), cuda(rng.standard_normal((T, H_I)).astype(np.float32))
        sel = M.misa_indexer_paged(iq, iw, keys, table, kbar, n, B, h, topk)
        o, lse = M.misa_kv4_attention(one, pool, table, n, idx=sel["idx"], acc=acc, want_lse=True)
        pl = host(pool)
        for t in range(T):
            pos = np.sort(host(sel["idx"])[t])
            pos = pos[pos >= 0]
            assert len(pos) == min(topk, nh[t])
            kk, vv = R.cache_rows(pl, table_h[t], pos, page, d)
            qq = host(one[t:t + 1].float())
            want, z, p = R.attend(qq, kk, vv, d ** -0.5)
            tol, e = R.attend_tolerance(qq, kk, vv, d ** -0.5, p, "bf16", 2.0 ** -11, 2.0 ** -36)
            assert np.all(np.abs(host(o[t].float()) - want[0]) <= tol[0])
            np.add.at(acc_ref[t], pos, p[:, 0].sum(0))
        assert np.all(np.abs(host(acc) - acc_ref) <= 1e-4 * acc_ref + 1e-6)

    for _ in range(3):
        step()
    keep, sink, recent = 200, 4, 16
    before_k, before_keys = host(pool).copy(), host(keys.float()).copy()
    idx, n2, acc2 = M.misa_evict_select(acc, n, keep, sink, recent, acc_out=torch.empty_like(acc))
    acc_h = host(acc)
    M.misa_kv4_compact(pool, table, idx, d)
    M.misa_keys_compact_paged(keys, table, idx)
    after, after_keys = host(pool), host(keys.float())
    for t in range(T):
        stay = np.array(R.evict(acc_h[t], int(nh[t]), keep, sink, recent))
        assert host(idx)[t][:len(stay)].tolist() == stay.tolist()
        j = np.arange(len(stay))
        for a, b in zip(R.cache_rows(before_k, table_h[t], stay, page, d), R.cache_rows(after, table_h[t], j, page, d)):
            assert np.array_equal(a, b)
        assert np.array_equal(before_keys[table_h[t, stay // page], stay % page], after_keys[table_h[t, j // page], j % page])
        acc_ref[t] = np.concatenate([acc_ref[t, stay], np.zeros(per * page - len(stay))])
    n.copy_(n2)
    nh = host(n2).astype(int)
    assert nh.tolist() == [200, 200, 200]
    acc.copy_(acc2)
    for _ in range(2):
        step()
    M.misa_device_check()


def test_graphs_captured_without_a_workspace_replay_at_once():
    """Two graphs of the same calls, captured one after the other on one stream, keep scratch of their own: they
    are replayed on two streams at once, after an eager call has taken more scratch."""
    M = lib()
    T, Hq, Hkv, d, page, cap, keep = 4, 16, 2, 128, 64, 2048, 1500
    gen = torch.Generator("cuda").manual_seed(5)
    randn = lambda *s: torch.randn(*s, device="cuda", generator=gen).bfloat16()  # noqa: E731
    table = torch.arange(T * cap // page, device="cuda", dtype=torch.int32).reshape(T, -1)
    n = torch.full((T,), cap, device="cuda", dtype=torch.int32)
    cu = torch.arange(T + 1, device="cuda", dtype=torch.int32) * cap
    zero = torch.zeros(T, device="cuda", dtype=torch.int32)
    cq, ck = (torch.tensor([0, x], device="cuda", dtype=torch.int32) for x in (300, 9000))
    idx = torch.stack([torch.randperm(cap, device="cuda", generator=gen)[:keep].sort().values for _ in range(T)]).int()

    def state():
        pool = M.misa_kv4_pool(T * cap // page, page, Hkv, d)
        M.misa_kv4_append(randn(T * cap, Hkv, d), randn(T * cap, Hkv, d), pool, table, cu, zero)
        return dict(pool=pool, q=randn(T, Hq, d), acc=torch.zeros(T, cap, device="cuda"), pq=randn(300, 4, d),
                    pk=randn(9000, 2, d), pv=randn(9000, 2, d))

    def run(s):
        out, lse = M.misa_kv4_attention(s["q"], s["pool"], table, n, acc=s["acc"], want_lse=True)
        pout, _ = M.misa_prompt_attention(s["pq"], s["pk"], s["pv"], cq, ck)
        M.misa_kv4_compact(s["pool"], table, idx, d)
        return out, lse, pout

    states = [state() for _ in range(2)]
    kept = [{k: s[k].clone() for k in ("pool", "acc")} for s in states]
    want = [(*run(s), s["pool"].clone(), s["acc"].clone()) for s in states]
    graphs, outs = [], []
    side = torch.cuda.Stream()
    for s in states:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            outs.append(run(s))
        graphs.append(g)
    with torch.cuda.stream(side):  # more scratch than the captured calls took
        big = randn(8, 64, d)
        wide = torch.arange(8 * cap // page, device="cuda", dtype=torch.int32).reshape(8, -1) % (T * cap // page)
        M.misa_kv4_attention(big, states[0]["pool"], wide, torch.full((8,), cap, device="cuda", dtype=torch.int32),
                             acc=torch.zeros(8, cap, device="cuda"))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        for s, k in zip(states, kept):
            for name in k:
                s[name].copy_(k[name])
        torch.cuda.synchronize()
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        for s, o, w in zip(states, outs, want):
            assert all(torch.equal(x, y) for x, y in zip((*o, s["pool"], s["acc"]), w))
    M.misa_device_check()


def test_calls_on_a_stream_beside_the_current_one():
    """Outputs and inputs of a call on another stream: the memory of neither is handed out again too early."""
    M = lib()
    T, Hq, Hkv, d, page, cap = 8, 16, 2, 128, 64, 4096
    gen = torch.Generator("cuda").manual_seed(9)
    randn = lambda *s: torch.randn(*s, device="cuda", generator=gen).bfloat16()  # noqa: E731
    table = torch.arange(T * cap // page, device="cuda", dtype=torch.int32).reshape(T, -1)
    pool = M.misa_kv4_pool(T * cap // page, page, Hkv, d)
    cu = torch.arange(T + 1, device="cuda", dtype=torch.int32) * cap
    zero, n = torch.zeros(T, device="cuda", dtype=torch.int32), torch.full((T,), cap, device="cuda", dtype=torch.int32)
    M.misa_kv4_append(randn(T * cap, Hkv, d), randn(T * cap, Hkv, d), pool, table, cu, zero)
    q = randn(T, Hq, d)
    pq, pk, pv = randn(2000, Hq, d), randn(2000, Hkv, d), randn(2000, Hkv, d)
    pc = torch.tensor([0, 2000], device="cuda", dtype=torch.int32)
    want = M.misa_kv4_attention(q, pool, table, n)[0].clone()
    pwant = M.misa_prompt_attention(pq, pk, pv, pc)[0].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    outs = []
    for _ in range(20):
        junk = torch.full((T, Hq, d), 3.0, device="cuda", dtype=torch.bfloat16)  # work on the current stream
        junk.mul_(2.0)
        del junk
        q1 = q.clone()
        side.wait_stream(torch.cuda.current_stream())
        o, _ = M.misa_kv4_attention(q1, pool, table, n, stream=side)
        p, _ = M.misa_prompt_attention(pq, pk, pv, pc, stream=side)
        del q1
        torch.full((T, Hq, d), float("nan"), device="cuda", dtype=torch.bfloat16)  # as large as q1 was
        outs.append((o, p))
    torch.cuda.current_stream().wait_stream(side)
    for o, p in outs:
        assert torch.equal(o, want) and torch.equal(p, pwant)
