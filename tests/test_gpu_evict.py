"""Thinning caches by summed attention weight: which tokens stay, and the caches closing up in place."""
import numpy as np
import pytest
import torch

import attention_ref as R
from gpu_common import host, lib

pytestmark = pytest.mark.gpu


def cuda(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def weights(rng, T, L, kind):
    if kind == "equal":
        return np.full((T, L), 0.25, np.float32)
    a = rng.exponential(1.0, (T, L)).astype(np.float32)
    if kind == "ties":
        a = np.floor(a * 2) / 2
    if kind == "odd":  # everything that is not an ordinary weight
        a[:, ::7] = -0.0
        a[:, 1::7] = 0.0
        a[:, 2::13] = np.inf
        a[:, 3::11] = np.nan
        a[:, 4::9] *= -1
        a[:, 5::17] = -np.inf
        a[:, 6::19] = 1e-42
    return a


@pytest.mark.parametrize("kind", ["plain", "ties", "odd", "equal"])
@pytest.mark.parametrize("lens,keep,sink,recent", [
    ([1, 0, 5, 100, 101, 102, 1000], 100, 4, 20),
    ([1023, 1024, 1025, 4097, 9000], 300, 0, 0),
    ([20000, 7, 12345], 5000, 64, 1000),
    ([500, 501, 40], 41, 1, 40),       # nothing but sinks and recents
    ([500, 3], 1, 0, 0),
    ([500, 300], 1, 0, 1),
    ([70000, 65536, 66000], 1025, 4, 7),
])
def test_the_tokens_that_stay(kind, lens, keep, sink, recent):
    M = lib()
    rng = np.random.default_rng(keep + len(lens))
    T, L = len(lens), max(lens)
    acc = weights(rng, T, L + 3, kind)
    n = np.array(lens, np.int32)
    out = torch.full((T, keep + 5), 9.0, device="cuda")
    idx, no, ao = M.misa_evict_select(cuda(acc), cuda(n), keep, sink, recent, acc_out=out)
    for t in range(T):
        want = R.evict(acc[t], lens[t], keep, sink, recent)
        assert int(no[t]) == len(want)
        assert host(idx)[t].tolist() == want + [-1] * (keep - len(want)), t
        assert np.array_equal(host(ao)[t, :len(want)], acc[t, want], equal_nan=True)
        assert np.all(host(ao)[t, len(want):] == 0)


@pytest.mark.parametrize("kind", ["plain", "odd", "equal"])
@pytest.mark.parametrize("lens,keep", [([40000, 32769], 17000), ([131072, 3, 65537], 2000), ([140000, 139999], 70000)])
def test_long_rows(kind, lens, keep):
    M = lib()
    rng = np.random.default_rng(keep)
    acc = weights(rng, len(lens), max(lens), kind)
    idx, no, ao = M.misa_evict_select(cuda(acc), cuda(np.array(lens, np.int32)), keep, 4, 33, want_acc=True)
    for t in range(len(lens)):
        want = R.evict(acc[t], lens[t], keep, 4, 33)
        assert int(no[t]) == len(want) and host(idx)[t].tolist() == want + [-1] * (keep - len(want))
        assert np.array_equal(host(ao)[t, :len(want)], acc[t, want], equal_nan=True)


def test_lengths_outside_the_row_and_limits():
    M = lib()
    acc = np.random.default_rng(1).random((3, 50)).astype(np.float32)
    idx, no, _ = M.misa_evict_select(cuda(acc), cuda(np.array([-3, 900, 50], np.int32)), 10, L=40)
    assert host(no).tolist() == [0, 10, 10]
    for t, n in enumerate((0, 40, 40)):
        want = R.evict(acc[t], n, 10, 0, 0)
        assert host(idx)[t].tolist() == want + [-1] * (10 - len(want))


@pytest.mark.parametrize("Hkv,d,page,lens,keep", [
    (2, 128, 16, [100, 37, 0, 64], 40),
    (3, 64, 48, [500, 499], 200),
    (8, 128, 64, [30000, 25000], 20000),   # many segments of rows, more than the GPU runs at once
])
def test_caches_close_up_in_place(Hkv, d, page, lens, keep):
    M = lib()
    rng = np.random.default_rng(keep)
    T, per = len(lens), -(-max(max(lens), keep) // page)
    total = T * per + 2
    table = rng.permutation(total)[:T * per].reshape(T, per).astype(np.int32)
    pool = rng.integers(0, 256, (total, Hkv, 2, page * 9 * d // 16), dtype=np.uint8)
    keys = rng.standard_normal((total, page, 128)).astype(np.float32)
    acc = rng.random((T, max(lens))).astype(np.float32)
    idx, no, _ = M.misa_evict_select(cuda(acc), cuda(np.array(lens, np.int32)), keep, 2, 5)
    pd, kd, kb = cuda(pool), cuda(keys), cuda(keys).bfloat16()
    kb0 = kb.clone()
    M.misa_kv4_compact(pd, cuda(table), idx, d)
    M.misa_keys_compact_paged(kd, cuda(table), idx)
    M.misa_keys_compact_paged(kb, cuda(table), idx)
    want, wk = pool.copy(), keys.copy()
    c0, s0 = R.views(pool, page, d)
    c1, s1 = R.views(want, page, d)
    order = torch.arange(total * page, device="cuda").view(total, page)
    src = host(order).copy()
    for t in range(T):
        pos = host(idx)[t][:int(no[t])]
        j = np.arange(len(pos))
        a, b = (table[t, pos // page], pos % page), (table[t, j // page], j % page)
        c1[b[0], :, :, b[1]], s1[b[0], :, :, b[1]] = c0[a[0], :, :, a[1]], s0[a[0], :, :, a[1]]
        wk[b] = keys[a]
        src[b] = host(order)[a]
    assert np.array_equal(host(pd), want)
    assert np.array_equal(host(kd), wk)
    assert torch.equal(kb, kb0.view(-1, 128)[cuda(src).view(-1)].view_as(kb))


def test_a_page_out_of_the_pool_stops_only_its_rows():
    M = lib()
    rng = np.random.default_rng(4)
    pool = rng.integers(0, 256, (6, 1, 2, 16 * 72), dtype=np.uint8)
    table = np.array([[3, 77, 1]], np.int32)
    idx = np.array([[0, 2, 17, 18, 33, 34, 47, -1]], np.int32)  # rows 17, 18 lie in the page that is not there
    pd = cuda(pool)
    M.misa_kv4_compact(pd, cuda(table), cuda(idx), 128)
    want = pool.copy()
    c0, s0 = R.views(pool, 16, 128)
    c1, s1 = R.views(want, 16, 128)
    for j, s in enumerate(idx[0]):
        if s >= 0 and s // 16 != 1:
            c1[3, :, :, j], s1[3, :, :, j] = c0[table[0, s // 16], :, :, s % 16], s0[table[0, s // 16], :, :, s % 16]
    assert np.array_equal(host(pd), want)


def test_eviction_captured():
    M = lib()
    rng = np.random.default_rng(5)
    acc, n = cuda(rng.random((2, 3000)).astype(np.float32)), cuda(np.array([3000, 1500], np.int32))
    table = cuda(np.arange(2 * 188, dtype=np.int32).reshape(2, 188))
    pool = cuda(rng.integers(0, 256, (376, 2, 2, 16 * 36), dtype=np.uint8))
    idx, no, ao = (torch.empty(2, 700, dtype=torch.int32, device="cuda"), torch.empty(2, dtype=torch.int32, device="cuda"),
                   torch.empty(2, 700, device="cuda"))

    ws = M.Workspace()

    def step(p):
        M.misa_evict_select(acc, n, 700, 4, 50, idx=idx, n_out=no, acc_out=ao)
        M.misa_kv4_compact(p, table, idx, 64, ws=ws)

    step(pool.clone())
    torch.cuda.synchronize()
    first = pool.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(first)
    acc.copy_(cuda(rng.random((2, 3000)).astype(np.float32)))
    first.copy_(pool)
    g.replay()
    torch.cuda.synchronize()
    got = [x.clone() for x in (idx, no, ao, first)]
    again = pool.clone()
    step(again)
    assert all(torch.equal(x, y) for x, y in zip(got, (idx, no, ao, again)))
