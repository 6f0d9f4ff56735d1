"""4-bit key and value caches on the GPU: the stored bytes against the format's definition, attention
over them against the formula in double precision."""
import numpy as np
import pytest
import torch

import attention_ref as R
from gpu_common import host, lib

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# Weights are rounded to fp16 scaled by 2^11 against the running maximum.  fp16 steps by 2^-24 below its
# normal range, so a small weight is off by at most 2^-25 2^-11 = 2^-36 of the largest one, itself at most 1.
FLOOR = 2.0 ** -36


def cuda(x, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(x)).cuda()
    return t if dtype is None else t.to(dtype)


def cum(lens):
    return np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)


def make_pool(rng, T, L, Hkv, d, page, spare=3):
    """A pool of random codes with scales between 2^-4 and 2^0 behind shuffled tables."""
    per = -(-L // page)
    total = T * per + spare
    pool = rng.integers(0, 256, (total, Hkv, 2, page * 9 * d // 16), dtype=np.uint8)
    scales = pool[..., page * d // 2:]
    scales[...] = (scales & 31) + 0x18
    table = rng.permutation(total)[:T * per].reshape(T, per).astype(np.int32)
    return pool, table


# ---- append and read ----------------------------------------------------------------------------------

@pytest.mark.parametrize("dtype,d,Hkv,page,lens,starts,kg,vg", [
    ("bf16", 128, 8, 64, [5, 0, 130, 1], [0, 3, 61, 1000], 1.0, 1.0),
    ("bf16", 64, 1, 16, [1], [0], 1.0, 0.125),
    ("f32", 128, 3, 48, [17, 33], [15, 0], 0.37, 1.9),
    ("f32", 64, 2, 32, [0, 1, 2, 31, 64], [7, 31, 32, 33, 0], 1.0, 0.01),
])
def test_append_stores_the_format_and_read_inverts_it(dtype, d, Hkv, page, lens, starts, kg, vg):
    M = lib()
    rng = np.random.default_rng(d + page + len(lens))
    S, L = len(lens), max(a + b for a, b in zip(lens, starts))
    pool, table = make_pool(rng, S, L, Hkv, d, page)
    rows = sum(lens) + 3  # rows behind the last sequence: neither read nor written
    cu = cum(lens) + 1    # and one before the first
    x = [rng.standard_normal((rows, Hkv, d)).astype(np.float32) * rng.choice([1e-3, 0.1, 1, 30], (rows, Hkv, d // 16)).repeat(16, -1)
         for _ in range(2)]
    for a in x:
        a[1, 0, :16] = 0.0                      # a block of zeros
        a[1, 0, 16:32] = [6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, -0.25, -0.75, -1.25, -1.75, -2.5, -3.5, -5, -0.0]  # ties
        a[1, 0, 32:48] = 1e-9                   # a scale that rounds to zero
        a[1, 0, 48:64] = np.array([1e6, -1e6, 1.0, 400.0] * 4)  # above the largest scale
    x = [host(cuda(a, DT[dtype]).float()) for a in x]
    k, v = (cuda(a, DT[dtype]) for a in x)
    k[0] = float("nan")
    v[rows - 1] = float("inf")
    pd, td = cuda(pool), cuda(table)
    M.misa_kv4_append(k, v, pd, td, cuda(cu), cuda(np.array(starts, np.int32)), k_scale=kg, v_scale=vg)
    want = pool.copy()
    codes, scales = R.views(want, page, d)
    packed = [R.pack(a, g) for a, g in zip(x, (kg, vg))]
    for b in range(S):
        for i in range(lens[b]):
            s, r = starts[b] + i, cu[b] + i
            for side in range(2):
                codes[table[b, s // page], :, side, s % page] = packed[side][0][r]
                scales[table[b, s // page], :, side, s % page] = packed[side][1][r]
    got = host(pd)
    gc, gs = R.views(got, page, d)
    # zeros compare as values: a code's sign on zero is not part of the format's meaning
    for g_, w_ in ((gc & 15, codes & 15), (gc >> 4, codes >> 4)):
        assert np.array_equal(np.where(g_ == 8, 0, g_), np.where(w_ == 8, 0, w_))
    assert np.array_equal(gs, scales)
    out = {}
    for kind in ("bf16", "f32"):
        kb, vb = (torch.full((rows, Hkv, d), 7.0, dtype=DT[kind], device="cuda") for _ in range(2))
        M.misa_kv4_read(pd, td, cuda(cu), cuda(np.array(starts, np.int32)), rows, d, dtype=DT[kind], k_scale=kg,
                        v_scale=vg, k=kb, v=vb)
        out[kind] = (host(kb.float()), host(vb.float()))
        for side, g in ((0, kg), (1, vg)):
            val = R.unpack(*packed[side]) * float(np.float32(g))
            # code x scale is exact; times g, and rounded to the output's type (half a step each)
            tol = (2.0 ** -24 if kind == "f32" else (0.0 if g in (1.0, 0.125) else 2.0 ** -8 + 2.0 ** -24)) * np.abs(val)
            mine = out[kind][side]
            assert np.all(np.abs(mine[1:-2] - val[1:-2]) <= tol[1:-2])
            assert np.all(mine[0] == 7) and np.all(mine[-2:] == 7), "rows of no sequence are left as they were"


def test_append_of_strided_rows_infinities_and_nan():
    M = lib()
    rng = np.random.default_rng(3)
    rows, Hq, Hkv, d, page = 21, 4, 2, 128, 16
    fused = cuda(rng.standard_normal((rows, (Hq + 2 * Hkv) * d)).astype(np.float32), torch.bfloat16)
    k = fused[:, Hq * d:(Hq + Hkv) * d].unflatten(1, (Hkv, d))
    v = fused[:, (Hq + Hkv) * d:].unflatten(1, (Hkv, d))
    k[2, 0, 5], k[2, 0, 20], k[2, 0, 40] = float("nan"), float("inf"), -float("inf")
    pools = [M.misa_kv4_pool(4, page, Hkv, d) for _ in range(2)]
    td, cu, st = cuda(np.array([[2, 0]], np.int32)), cuda(cum([rows])), cuda(np.zeros(1, np.int32))
    M.misa_kv4_append(k, v, pools[0], td, cu, st)
    M.misa_kv4_append(k.contiguous(), v.contiguous(), pools[1], td, cu, st)
    assert torch.equal(*pools)
    kb, _ = M.misa_kv4_read(pools[0], td, cu, st, rows, d)
    assert kb[2, 0, 5] == 0 and kb[2, 0, 20] == 6 * 448 and kb[2, 0, 40] == -6 * 448
    assert torch.isfinite(kb.float()).all()


def test_rows_outside_the_pages_are_skipped():
    M = lib()
    Hkv, d, page = 2, 64, 16
    pool = torch.full((3, Hkv, 2, page * 9 * d // 16), 0x31, dtype=torch.uint8, device="cuda")
    before = pool.clone()
    table = cuda(np.array([[1, 99], [-5, 2]], np.int32))
    k = torch.randn(40, Hkv, d, device="cuda").bfloat16()
    cu, start = cuda(np.array([0, 20, 40], np.int32)), cuda(np.array([30, 10], np.int32))
    M.misa_kv4_append(k, k, pool, table, cu, start)  # positions 30..49 (pages 1.., 99, none) and 10..29 (-5, 2)
    assert torch.equal(pool[0], before[0]), "a page no table names"
    kb, vb = M.misa_kv4_read(pool, table, cu, start, 40, d, dtype=torch.float32)
    assert (kb[:20] == 0).all() and (kb[20:26] == 0).all() and (vb[20:26] == 0).all()
    assert (kb[26:] != 0).any(dim=-1).all()
    assert torch.equal(pool[1], before[1]), "no position of the call lies in page 1"


# ---- attention ------------------------------------------------------------------------------------------

def check_attention(M, rng, T, lens, Hq, Hkv, d, page, dtype, pick=None, acc=False, kg=1.0, vg=1.0, scale=None,
                    spread=1.0, L=None):
    cap = max(max(lens), 1)
    pool, table = make_pool(rng, T, cap, Hkv, d, page)
    # what lies behind a prefix is garbage: NaN scales in every row from n_t on
    _, scales = R.views(pool, page, d)
    for t in range(T):
        for s in range(max(0, lens[t]), table.shape[1] * page):
            scales[table[t, s // page], :, :, s % page] = 0x7f
    q = cuda((rng.standard_normal((T, Hq, d)) * spread).astype(np.float32), DT[dtype])
    a0 = rng.random((T, cap)).astype(np.float32)
    accd = cuda(a0) if acc else None
    idx = None
    if pick is not None:
        idx = np.full((T, pick), -1, np.int32)
        for t in range(T):
            n = max(0, lens[t])
            got = rng.permutation(n)[:pick]
            where = rng.permutation(pick)[:len(got)]  # empty slots anywhere
            idx[t, where] = got
        if pick > 2:
            idx[0, idx[0] < 0] = cap + 5 if cap + 5 > lens[0] else -1  # past the prefix: an empty slot too
    out, lse = M.misa_kv4_attention(q, cuda(pool), cuda(table), cuda(np.array(lens, np.int32)),
                                    idx=None if idx is None else cuda(idx), L=L, scale=scale, k_scale=kg, v_scale=vg,
                                    acc=accd, want_lse=True)
    out, lse, qh = host(out.float()), host(lse), host(q.float()).astype(np.float64)
    sc = (d ** -0.5 if scale is None else scale)
    for t in range(T):
        n = min(max(0, lens[t]), cap if L is None else L)
        pos = np.arange(n) if idx is None else np.array([i for i in idx[t] if 0 <= i < n], int)
        if not len(pos):
            assert np.all(out[t] == 0) and np.all(np.isneginf(lse[t]))
            if acc:
                assert np.array_equal(host(accd)[t], a0[t])
            continue
        k, v = R.cache_rows(pool, table[t], pos, page, d)
        k, v = k * float(np.float32(kg)), v * float(np.float32(vg))
        want, z, p = R.attend(qh[t:t + 1], k, v, sc)
        # weights: fp16 for bf16 outputs (half a step, 2^-11), two fp16 parts for fp32 ones
        tol, e = R.attend_tolerance(qh[t:t + 1], k, v, sc, p, dtype, 2.0 ** -11 if dtype == "bf16" else 2.0 ** -21,
                                    FLOOR)
        assert np.all(np.abs(out[t] - want[0]) <= tol[0]), (t, (np.abs(out[t] - want[0]) / tol[0]).max())
        ltol = e + 2.0 ** -23 * np.abs(z[0]) + 2.0 ** -24 * max(16, len(pos)) + 2.0 ** -20
        assert np.all(np.abs(lse[t] - z[0]) <= ltol)
        if acc:
            ref = a0[t].astype(np.float64)
            np.add.at(ref, pos, p[:, 0].sum(0))
            add = ref - a0[t]
            atol = add * (2 * ltol.max() + 2.0 ** -20 + Hq * 2.0 ** -24) + 2.0 ** -23 * np.abs(ref)
            assert np.all(np.abs(host(accd)[t] - ref) <= atol)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,Hq,Hkv,page,lens", [
    (128, 8, 8, 64, [1, 15, 16, 17, 63, 64, 65, 200]),     # no sharing; lengths around a tile and a page
    (128, 32, 4, 16, [700, 0, 1, 333]),                    # 8 heads on one, an empty prefix
    (64, 6, 2, 48, [129, 50]),                             # groups of 3, pages that are no power of two
    (128, 11, 1, 32, [513, 64]),                           # 11 heads on one: two column blocks
    (64, 40, 2, 128, [300]),                               # 20 heads on one: two blocks of 16
    (128, 128, 1, 64, [100, 2000]),                        # 128 heads on one
])
def test_attention_over_the_whole_prefix(dtype, d, Hq, Hkv, page, lens):
    rng = np.random.default_rng(len(lens) * d + Hq)
    check_attention(lib(), rng, len(lens), lens, Hq, Hkv, d, page, dtype, acc=Hq % 2 == 0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("pick,lens,Hq,Hkv,d", [
    (1, [1, 40, 0], 8, 1, 128),
    (37, [200, 20, 1000], 12, 4, 64),
    (130, [129, 131, 5], 32, 2, 128),
    (512, [4000], 64, 8, 128),
])
def test_attention_over_selected_tokens(dtype, pick, lens, Hq, Hkv, d):
    rng = np.random.default_rng(pick)
    check_attention(lib(), rng, len(lens), lens, Hq, Hkv, d, 32, dtype, pick=pick, acc=True)


def test_attention_scales_sharp_logits_and_lengths_past_the_limit():
    M = lib()
    rng = np.random.default_rng(9)
    check_attention(M, rng, 2, [300, 77], 8, 2, 128, 16, "bf16", kg=0.25, vg=3.7, scale=0.31, acc=True)
    check_attention(M, rng, 2, [300, 77], 8, 2, 64, 16, "f32", kg=1.7, vg=0.01)
    check_attention(M, rng, 2, [900, 901], 16, 2, 128, 64, "bf16", spread=20.0)  # one token takes nearly all
    check_attention(M, rng, 2, [900, 901], 16, 2, 128, 64, "bf16", spread=1e-3)  # nearly uniform
    check_attention(M, rng, 3, [300, -4, 77], 8, 2, 128, 16, "f32", L=100)       # above L counts as L, below 1 as 0
    check_attention(M, rng, 1, [40000], 8, 1, 128, 64, "bf16", acc=True)         # many pieces of one head
    check_attention(M, rng, 1, [40000], 4, 1, 64, 64, "f32")


def test_attention_of_more_queries_than_one_launch_takes():
    rng = np.random.default_rng(11)
    lens = rng.integers(0, 40, 1030).tolist()
    check_attention(lib(), rng, len(lens), lens, 2, 1, 64, 16, "bf16", acc=True)


@pytest.mark.parametrize("pick", [None, 300])
@pytest.mark.parametrize("d,Hq,Hkv", [(128, 16, 2), (64, 36, 3)])
def test_many_heads_of_a_few_pieces_each(pick, d, Hq, Hkv):
    """More heads than one wave of CTAs, cut into pieces by the split of the tokens."""
    rng = np.random.default_rng(Hq)
    lens = rng.integers(0, 1500, 38).tolist() + [4096, 0]
    check_attention(lib(), rng, len(lens), lens, Hq, Hkv, d, 64, "bf16", pick=pick, acc=True)


def test_a_token_named_twice_counts_twice():
    M = lib()
    rng = np.random.default_rng(12)
    pool, table = make_pool(rng, 1, 64, 2, 128, 16)
    q = cuda(rng.standard_normal((1, 8, 128)).astype(np.float32))
    pos = np.array([3, 50, 3, 7, 3], np.int32)
    acc = torch.zeros(1, 64, device="cuda")
    out, lse = M.misa_kv4_attention(q, cuda(pool), cuda(table), cuda(np.array([64], np.int32)), idx=cuda(pos[None]),
                                    acc=acc, want_lse=True)
    k, v = R.cache_rows(pool, table[0], pos, 16, 128)
    want, z, p = R.attend(host(q).astype(np.float64), k, v, 128 ** -0.5)
    tol, e = R.attend_tolerance(host(q), k, v, 128 ** -0.5, p, "f32", 2.0 ** -21, FLOOR)
    assert np.all(np.abs(host(out)[0] - want[0]) <= tol[0])
    ref = np.zeros(64)
    np.add.at(ref, pos, p[:, 0].sum(0))
    assert np.all(np.abs(host(acc)[0] - ref) <= ref * (4 * e + 2.0 ** -18))


def test_a_query_that_is_not_finite_stays_so_and_stays_alone():
    M = lib()
    rng = np.random.default_rng(13)
    pool, table = make_pool(rng, 2, 100, 2, 128, 16)
    q = cuda(rng.standard_normal((2, 8, 128)).astype(np.float32), torch.bfloat16)
    n = cuda(np.array([100, 90], np.int32))
    good, _ = M.misa_kv4_attention(q, cuda(pool), cuda(table), n)
    q[0, 1, 7] = float("nan")
    bad, lse = M.misa_kv4_attention(q, cuda(pool), cuda(table), n, want_lse=True)
    assert torch.isnan(bad[0, 1].float()).all() and torch.isnan(lse[0, 1])
    rest = [h for h in range(8) if h != 1]
    assert torch.equal(bad[0, rest], good[0, rest]) and torch.equal(bad[1], good[1])


def test_pages_out_of_the_pool_are_left_out():
    M = lib()
    rng = np.random.default_rng(14)
    pool, table = make_pool(rng, 1, 128, 2, 64, 16)
    bad = table.copy()
    bad[0, 2], bad[0, 7] = 10 ** 6, -3
    q = cuda(rng.standard_normal((1, 4, 64)).astype(np.float32))
    n = cuda(np.array([120], np.int32))
    a, la = M.misa_kv4_attention(q, cuda(pool), cuda(bad), n, want_lse=True)
    keep = np.array([s for s in range(120) if s // 16 not in (2, 7)], np.int32)
    k, v = R.cache_rows(pool, table[0], keep, 16, 64)
    want, z, p = R.attend(host(q).astype(np.float64), k, v, 0.125)
    tol, e = R.attend_tolerance(host(q), k, v, 0.125, p, "f32", 2.0 ** -21, FLOOR)
    assert np.all(np.abs(host(a)[0] - want[0]) <= tol[0])
    b, _ = M.misa_kv4_attention(q, cuda(pool), cuda(bad), n, idx=cuda(np.arange(120, dtype=np.int32)[None]))
    assert np.all(np.abs(host(b)[0] - want[0]) <= tol[0])


def test_attention_is_the_same_from_run_to_run():
    M = lib()
    rng = np.random.default_rng(15)
    pool, table = make_pool(rng, 4, 3000, 4, 128, 64)
    q = cuda(rng.standard_normal((4, 16, 128)).astype(np.float32), torch.bfloat16)
    n = cuda(np.array([3000, 2999, 1000, 64], np.int32))
    pd, td = cuda(pool), cuda(table)
    got = []
    for _ in range(3):
        acc = torch.zeros(4, 3000, device="cuda")
        got.append((*M.misa_kv4_attention(q, pd, td, n, acc=acc, want_lse=True), acc))
    for g in got[1:]:
        assert all(torch.equal(x, y) for x, y in zip(g, got[0]))


def test_attention_captured_and_on_two_streams():
    """A captured call follows what its inputs hold at replay; calls on two streams do not share scratch."""
    M = lib()
    rng = np.random.default_rng(16)
    pool, table = make_pool(rng, 2, 2000, 2, 128, 64)
    pd, td = cuda(pool), cuda(table)
    q = cuda(rng.standard_normal((2, 16, 128)).astype(np.float32), torch.bfloat16)
    n = cuda(np.array([2000, 5], np.int32))
    acc = torch.zeros(2, 2000, device="cuda")
    ws = M.Workspace()
    out, lse = torch.empty_like(q), torch.empty(2, 16, device="cuda")
    call = lambda **kw: M.misa_kv4_attention(q, pd, td, n, out=out, lse=lse, acc=acc, **kw)  # noqa: E731
    call(ws=ws)  # the workspace is grown before the capture
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(ws=ws)
    n.copy_(cuda(np.array([7, 1999], np.int32)))
    q.mul_(0.5)
    acc.zero_()
    g.replay()
    torch.cuda.synchronize()
    got = [x.clone() for x in (out, lse, acc)]
    acc.zero_()
    call()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, (out, lse, acc)))
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for i in range(6):
        s = streams[i % 2]
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            outs.append(M.misa_kv4_attention(q, pd, td, n, want_lse=True))
    torch.cuda.synchronize()
    for o, z in outs:
        assert torch.equal(o, out) and torch.equal(z, lse)


def test_a_pool_past_four_gigabytes():
    """Byte offsets of the last pages need more than 32 bits."""
    M = lib()
    rng = np.random.default_rng(17)
    Hkv, d, page, L = 8, 128, 64, 200
    per = Hkv * 2 * page * 72
    total = (5 << 30) // per
    pool = torch.zeros(total, Hkv, 2, page * 72, dtype=torch.uint8, device="cuda")
    table = np.array([[total - 1, total - 3, 1, total - 2]], np.int32)
    k, v = (torch.randn(L, Hkv, d, device="cuda").bfloat16() for _ in range(2))
    cu, start = cuda(np.array([0, L], np.int32)), cuda(np.zeros(1, np.int32))
    M.misa_kv4_append(k, v, pool, cuda(table), cu, start)
    small = M.misa_kv4_pool(4, page, Hkv, d)
    st = cuda(np.array([[3, 1, 0, 2]], np.int32))
    M.misa_kv4_append(k, v, small, st, cu, start)
    q = cuda(rng.standard_normal((1, 32, d)).astype(np.float32), torch.bfloat16)
    n = cuda(np.array([L], np.int32))
    assert torch.equal(M.misa_kv4_attention(q, pool, cuda(table), n)[0], M.misa_kv4_attention(q, small, st, n)[0])
    idx = cuda(rng.permutation(L)[None, :90].astype(np.int32))
    assert torch.equal(M.misa_kv4_attention(q, pool, cuda(table), n, idx=idx)[0],
                       M.misa_kv4_attention(q, small, st, n, idx=idx)[0])
    a, b = M.misa_kv4_read(pool, cuda(table), cu, start, L, d), M.misa_kv4_read(small, st, cu, start, L, d)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
