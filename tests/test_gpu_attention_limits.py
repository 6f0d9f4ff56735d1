"""The attention calls in forms that a serving loop gives them beside the plain ones: lengths updated in place,
sums of weights narrower than the page table, values that are not finite beside segments without keys, and more
weights than one launch keeps."""
import numpy as np
import pytest
import torch

import attention_ref as R
from gpu_common import host, lib

pytestmark = pytest.mark.gpu


def cuda(x, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(x)).cuda()
    return t if dtype is None else t.to(dtype)


@pytest.mark.parametrize("lens,keep", [
    ([1000, 0, 300, 301, -5, 4000], 300),            # one CTA a row
    ([20000, 7, 12345, 5000, 5001, 32768] * 9, 5000),   # a cluster a row, more rows than run at once
    ([140000, 100, 70001], 70000),
])
def test_lengths_updated_in_place(lens, keep):
    M = lib()
    rng = np.random.default_rng(keep)
    T, L = len(lens), max(lens)
    acc = cuda(rng.random((T, L)).astype(np.float32))
    n = cuda(np.array(lens, np.int32))
    want = M.misa_evict_select(acc, n, keep, 3, 40, want_acc=True)
    assert torch.equal(want[1], n.clamp(0, keep))
    for t in (0, T - 1):
        assert host(want[0])[t, :int(want[1][t])].tolist() == R.evict(host(acc)[t], lens[t], keep, 3, 40)
    for _ in range(5):
        m = n.clone()
        got = M.misa_evict_select(acc, m, keep, 3, 40, n_out=m, want_acc=True)
        assert got[1] is m and all(torch.equal(x, y) for x, y in zip(got, want))


def serving_state(M, lens, page, per, Hkv, d, seed):
    """Caches of these lengths behind shuffled tables of `per` pages a sequence."""
    gen = torch.Generator("cuda").manual_seed(seed)
    T = len(lens)
    table = torch.randperm(T * per, device="cuda", generator=gen).int().view(T, per)
    pool = M.misa_kv4_pool(T * per, page, Hkv, d)
    cu = cuda(np.concatenate([[0], np.cumsum(lens)]).astype(np.int32))
    k, v = (torch.randn(sum(lens), Hkv, d, device="cuda", generator=gen).bfloat16() for _ in range(2))
    M.misa_kv4_append(k, v, pool, table, cu, cuda(np.zeros(T, np.int32)))
    return pool, table, cuda(np.array(lens, np.int32)), gen


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("selected", [False, True])
def test_tokens_appended_after_an_eviction_are_attended_to(wide, selected):
    """Summed weights that end before the table does change nothing in the attention of later tokens."""
    M = lib()
    Hq, Hkv, d, page, per, keep = 8, 2, 128, 16, 4, 50
    pool, table, n, gen = serving_state(M, [60, 40, 64], page, per, Hkv, d, 3)
    T = 3
    acc = torch.rand(T, per * page, device="cuda", generator=gen)
    room = torch.empty_like(acc) if wide else None
    idx, n, acc = M.misa_evict_select(acc, n, keep, 2, 9, acc_out=room, want_acc=not wide)
    M.misa_kv4_compact(pool, table, idx, d)
    assert tuple(acc.shape) == (T, per * page if wide else keep)
    one = torch.arange(T + 1, device="cuda", dtype=torch.int32)
    full = torch.zeros(T, per * page, device="cuda")
    full[:, :acc.shape[1]] = acc
    for step in range(9):
        k, v = (torch.randn(T, Hkv, d, device="cuda", generator=gen).bfloat16() for _ in range(2))
        M.misa_kv4_append(k, v, pool, table, one, n)
        n.add_(1)
        q = torch.randn(T, Hq, d, device="cuda", generator=gen).bfloat16()
        pick = None
        if selected:  # the newest token first
            pick = (n[:, None] - 1 - 7 * torch.arange(6, device="cuda", dtype=torch.int32)[None]).int().contiguous()
        want, lse = M.misa_kv4_attention(q, pool, table, n, idx=pick, acc=full, want_lse=True)
        bare, _ = M.misa_kv4_attention(q, pool, table, n, idx=pick)
        out, z = M.misa_kv4_attention(q, pool, table, n, idx=pick, acc=acc, want_lse=True)
        assert torch.equal(out, want) and torch.equal(z, lse) and torch.equal(bare, want), step
        assert torch.equal(acc, full[:, :acc.shape[1]]), step
    sums = (full.sum(1) - full[:, :keep].sum(1))
    assert (sums[[0, 2]] > 0).all(), "tokens past the sums' columns were attended to"


@pytest.mark.parametrize("junk", [float("inf"), float("nan")])
@pytest.mark.parametrize("d,Hq,Hkv,S,longest", [
    (64, 4, 2, 400, 128),    # a block a prompt: the guards are prompts ahead of the outputs
    (128, 3, 1, 400, 128),
    (64, 3, 3, 260, 300),    # both tiles, and prompts that one tile has alone
    (128, 2, 1, 700, 40),
])
def test_values_that_are_not_finite_in_neighbouring_prompts(junk, d, Hq, Hkv, S, longest):
    """Short prompts share CTAs, some of them without a key: the rows that see such a value, and only they, have it."""
    M = lib()
    rng = np.random.default_rng(S + d)
    keys = rng.integers(1, longest + 1, S)
    queries = keys.copy()
    for b in range(S):  # one to four prompts of ten that see nothing, one after another
        if b % 10 in ((2,), (2, 3), (2, 3, 4), (2, 3, 4, 5))[b // 10 % 4]:
            keys[b] = 0
    cu_q, cu_k = (np.concatenate([[0], np.cumsum(x)]).astype(np.int32) for x in (queries, keys))
    q = cuda(rng.standard_normal((cu_q[-1], Hq, d)).astype(np.float32), torch.bfloat16)
    k, v = (cuda(rng.standard_normal((cu_k[-1], Hkv, d)).astype(np.float32), torch.bfloat16) for _ in range(2))
    args = (cuda(cu_q), cuda(cu_k))
    good, gl = M.misa_prompt_attention(q, k, v, *args, want_lse=True)
    assert torch.isfinite(good.float()).all()
    want = good.clone()
    for b in range(S):
        if keys[b] == 0 or b % 7 == 0:
            continue
        at, e, h = int(rng.integers(keys[b])), int(rng.integers(d)), int(rng.integers(Hkv))
        v[cu_k[b] + at, h, e] = junk
        G = Hq // Hkv
        want[cu_q[b] + at:cu_q[b + 1], h * G:(h + 1) * G, e] = junk
    for _ in range(10):
        out, lse = M.misa_prompt_attention(q, k, v, *args, want_lse=True)
        assert torch.equal(torch.nan_to_num(out.float(), nan=-7e9, posinf=7e9), torch.nan_to_num(want.float(), nan=-7e9, posinf=7e9))
        assert torch.equal(lse, gl)
    M.misa_device_check()


@pytest.mark.parametrize("T,Hkv,d,page,L,keep", [
    (1, 1, 64, 16, 60000, 59000),     # rows move a little: every segment's place is read by its neighbour
    (1, 8, 128, 64, 40000, 39990),
    (24, 2, 128, 32, 9000, 8000),     # more segments than run at once, of many sequences
])
def test_closing_up_where_every_segment_waits_for_its_neighbours(T, Hkv, d, page, L, keep):
    M = lib()
    gen = torch.Generator("cuda").manual_seed(keep)
    per = -(-L // page)
    table = torch.randperm(T * per, device="cuda", generator=gen).int().view(T, per)
    pool = torch.randint(0, 256, (T * per, Hkv, 2, page * 9 * d // 16), device="cuda", dtype=torch.uint8, generator=gen)
    keys = torch.randn(T * per, page, 128, device="cuda", generator=gen)
    drop = torch.rand(T, L, device="cuda", generator=gen).argsort(1)[:, :L - keep]
    stay = torch.ones(T, L, dtype=torch.bool, device="cuda").scatter_(1, drop, False)
    idx = stay.nonzero()[:, 1].view(T, keep).int().contiguous()

    def split(p):
        a, b = p[..., :page * d // 2].unflatten(-1, (page, d // 2)), p[..., page * d // 2:].unflatten(-1, (page, d // 16))
        return [x[table.long()].permute(0, 1, 4, 2, 3, 5).reshape(T, per * page, -1) for x in (a, b)]

    before, kb = split(pool), keys[table.long()].view(T, per * page, 128)
    for _ in range(2):  # the closed-up cache closes up once more
        M.misa_kv4_compact(pool, table, idx, d)
        after = split(pool)
        for got, old in zip(after, before):
            for t in range(T):
                assert torch.equal(got[t, :keep], old[t, idx[t].long()]) and torch.equal(got[t, keep:], old[t, keep:])
        before = after
    M.misa_keys_compact_paged(keys, table, idx)
    got = keys[table.long()].view(T, per * page, 128)
    for t in range(T):
        assert torch.equal(got[t, :keep], kb[t, idx[t].long()]) and torch.equal(got[t, keep:], kb[t, keep:])
    M.misa_device_check()


@pytest.mark.parametrize("selected", [False, True])
def test_more_weights_than_one_launch_keeps(selected):
    """Logits past 1 GiB go in several launches: every query's output and sums are its own."""
    M = lib()
    rng = np.random.default_rng(8)
    T, Hq, d, page, L = 40, 128, 64, 64, 65536
    pool, one, _, gen = serving_state(M, [L], page, L // page, 1, d, 8)
    table = one.expand(T, -1).contiguous()  # one sequence, read by every query
    q = torch.randn(T, Hq, d, device="cuda", generator=gen).bfloat16()
    n = cuda(rng.integers(1, L + 1, T).astype(np.int32))
    n[0], n[31], n[32], n[39] = L, 1000, L, 0
    pick = None
    if selected:
        pick = torch.stack([torch.randperm(L, device="cuda", generator=gen) for _ in range(T)]).int()
    acc = torch.zeros(T, L, device="cuda")
    out, lse = M.misa_kv4_attention(q, pool, table, n, idx=pick, acc=acc, want_lse=True)
    for t in (0, 1, 30, 31, 32, 33, 39):  # alone: cut into other pieces, so equal up to rounding
        a = torch.zeros(1, L, device="cuda")
        o, z = M.misa_kv4_attention(q[t:t + 1], pool, one, n[t:t + 1].clone(), idx=None if pick is None else pick[t:t + 1],
                                    acc=a, want_lse=True)
        # weights in fp16 (2^-11 of sums of |v| below 1, either way), rounded to bf16 at the end (2^-8, either way);
        # the sum of a lane's weights takes up to 2^8 additions of 2^-24, either way, its exponentials add 2^-19
        assert (out[t].float() - o[0].float()).abs().max() <= 2 * 2.0 ** -8 * o.float().abs().max() + 2.0 ** -10
        both = torch.isinf(z[0]) & torch.isinf(lse[t])
        assert ((lse[t] - z[0]).abs() <= 2.0 ** -16 * z[0].abs() + 2.0 ** -14)[~both].all()
        assert (acc[t] - a[0]).abs().max() <= 2.0 ** -14 * a.max() and (acc[t, int(n[t]):] == 0).all()
        assert abs(float(acc[t].double().sum()) - (Hq if int(n[t]) else 0)) <= 2.0 ** -14 * Hq


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,Hq,Hkv,pick", [(128, 16, 2, None), (64, 12, 4, None), (128, 8, 1, 70), (64, 32, 2, 130)])
@pytest.mark.parametrize("top,kg,vg", [
    (0x07, 2.0 ** 9, 2.0 ** 8),      # zeros and the numbers below e4m3's normal range alone
    (0x10, 100.0, 37.0),             # both sides of its border
    (0x40, 0.4, 1.0),                # zero to 2
])
def test_attention_over_scales_below_the_normal_range(dtype, d, Hq, Hkv, pick, top, kg, vg):
    M = lib()
    rng = np.random.default_rng(top + d)
    page, lens = 32, [300, 1, 129]
    T, per = len(lens), 10
    pool = rng.integers(0, 256, (T * per, Hkv, 2, page * 9 * d // 16), dtype=np.uint8)
    _, scales = R.views(pool, page, d)
    scales[...] = rng.integers(0, top + 1, scales.shape)
    table = rng.permutation(T * per).reshape(T, per).astype(np.int32)
    q = cuda(rng.standard_normal((T, Hq, d)).astype(np.float32), torch.bfloat16 if dtype == "bf16" else None)
    idx = None
    if pick:
        idx = np.full((T, pick), -1, np.int32)
        for t, n in enumerate(lens):
            got = rng.permutation(n)[:pick]
            idx[t, :len(got)] = got
    out, lse = M.misa_kv4_attention(q, cuda(pool), cuda(table), cuda(np.array(lens, np.int32)),
                                    idx=None if idx is None else cuda(idx), k_scale=kg, v_scale=vg, want_lse=True)
    for t, n in enumerate(lens):
        pos = np.arange(n) if idx is None else idx[t][idx[t] >= 0]
        k, v = R.cache_rows(pool, table[t], pos, page, d)
        k, v = k * float(np.float32(kg)), v * float(np.float32(vg))
        qh = host(q[t:t + 1].float()).astype(np.float64)
        want, z, p = R.attend(qh, k, v, d ** -0.5)
        # weights: fp16 for bf16 outputs (half a step, 2^-11), two fp16 parts for fp32 ones; fp16 steps by 2^-24
        # below its normal range, of weights scaled by 2^11 against the largest: 2^-36
        tol, e = R.attend_tolerance(qh, k, v, d ** -0.5, p, dtype, 2.0 ** -11 if dtype == "bf16" else 2.0 ** -21, 2.0 ** -36)
        assert np.all(np.abs(host(out[t].float()) - want[0]) <= tol[0])
        assert np.all(np.abs(host(lse[t]) - z[0]) <= e + 2.0 ** -23 * np.abs(z[0]) + 2.0 ** -24 * max(16, len(pos)) + 2.0 ** -20)


def test_calls_with_given_outputs_and_workspace_allocate_nothing():
    """Neither through the caching allocator nor beside it, once each kernel has run."""
    M = lib()
    T, Hq, Hkv, d, page, per, keep = 4, 16, 2, 128, 64, 40, 1500
    pool, table, n, gen = serving_state(M, [per * page] * T, page, per, Hkv, d, 4)
    cap = per * page
    rows = 1000
    pq, pk, pv = (torch.randn(rows, h, d, device="cuda", generator=gen).bfloat16() for h in (Hq, Hkv, Hkv))
    cu, zero = cuda(np.array([0, 10, 700, rows], np.int32)), cuda(np.zeros(3, np.int32))
    keys = torch.randn(T * per, page, 128, device="cuda", generator=gen).bfloat16()
    acc, acc2 = torch.zeros(T, cap, device="cuda"), torch.zeros(T, cap, device="cuda")
    q, idx = torch.randn(T, Hq, d, device="cuda", generator=gen).bfloat16(), torch.zeros(T, keep, dtype=torch.int32, device="cuda")
    pout, plse, out, lse = torch.empty_like(pq), torch.empty(rows, Hq, device="cuda"), torch.empty_like(q), torch.empty(T, Hq, device="cuda")
    kb, vb = torch.empty_like(pk), torch.empty_like(pv)
    ws = M.Workspace()

    def step():
        M.misa_prompt_attention(pq, pk, pv, cu, out=pout, lse=plse, ws=ws)
        M.misa_kv4_append(pk, pv, pool, table[:3], cu, zero)
        M.misa_kv4_read(pool, table[:3], cu, zero, rows, d, k=kb, v=vb)
        M.misa_kv4_attention(q, pool, table, n, out=out, lse=lse, acc=acc, ws=ws)
        M.misa_kv4_attention(q, pool, table, n, idx=idx, out=out, ws=ws)
        M.misa_evict_select(acc, n, keep, 4, 50, idx=idx, n_out=n, acc_out=acc2)
        M.misa_kv4_compact(pool, table, idx, d, ws=ws)
        M.misa_keys_compact_paged(keys, table, idx, ws=ws)

    for _ in range(2):
        step()
    torch.cuda.synchronize()
    before = torch.cuda.memory_stats()["allocation.all.allocated"], torch.cuda.mem_get_info()[0]
    for _ in range(3):
        step()
    torch.cuda.synchronize()
    assert (torch.cuda.memory_stats()["allocation.all.allocated"], torch.cuda.mem_get_info()[0]) == before


def test_a_graph_replays_after_its_workspace_has_grown():
    """What a graph was captured with stays its own when a later, larger call replaces the workspace's buffer."""
    M = lib()
    Hq, Hkv, d, page, per = 16, 2, 128, 64, 16
    pool, table, n, gen = serving_state(M, [per * page - 5, 700], page, per, Hkv, d, 9)
    q = torch.randn(2, Hq, d, device="cuda", generator=gen).bfloat16()
    acc, out, lse = torch.zeros(2, per * page, device="cuda"), torch.empty_like(q), torch.empty(2, Hq, device="cuda")
    ws = M.Workspace()
    call = lambda w: M.misa_kv4_attention(q, pool, table, n, out=out, lse=lse, acc=acc, ws=w)  # noqa: E731
    call(ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(ws)
    acc.zero_()
    call(M.Workspace())
    want = [x.clone() for x in (out, lse, acc)]
    size = ws.buf.numel()
    wide = torch.randn(200, 64, d, device="cuda", generator=gen).bfloat16()
    rows = table[:1].expand(200, -1).contiguous()
    M.misa_kv4_attention(wide, pool, rows, n[:1].expand(200).contiguous(), acc=torch.zeros(200, per * page, device="cuda"), ws=ws)
    assert ws.buf.numel() > size
    torch.cuda.synchronize()
    others = [torch.full((size,), 0x5a, dtype=torch.uint8, device="cuda") for _ in range(4)]  # what a freed buffer would serve
    for _ in range(3):
        acc.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip((out, lse, acc), want))
        assert all((x == 0x5a).all() for x in others)
