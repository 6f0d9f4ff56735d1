"""Causal attention of packed prompts against the formula in double precision."""
import numpy as np
import pytest
import torch

import attention_ref as R
from gpu_common import host, lib

pytestmark = pytest.mark.gpu


def cuda(x, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(x)).cuda()
    return t if dtype is None else t.to(dtype)


def cum(lens):
    return np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)


def check(M, q, k, v, cu_q, cu_k, out, lse, scale, heads=None, rows=None):
    """Every row of every sequence (or a spread of `rows` of each) against the formula."""
    d = q.shape[-1]
    qh, kh, vh = (host(x.float()) for x in (q, k, v))
    o, z = host(out.float()), host(lse)
    for b in range(len(cu_q) - 1):
        q0, q1, k0, k1 = cu_q[b], cu_q[b + 1], cu_k[b], cu_k[b + 1]
        m, l = q1 - q0, k1 - k0
        if m == 0:
            continue
        at = np.arange(m) if rows is None or m <= rows else np.unique(np.linspace(0, m - 1, rows).astype(int))
        seen = np.arange(l)[None] <= (at + l - m)[:, None]
        want, lw, p = R.attend(qh[q0 + at], kh[k0:k1], vh[k0:k1], scale, seen)
        # weights are rounded to bf16 (half a step, 2^-8) for the product with V
        tol, e = R.attend_tolerance(qh[q0 + at], kh[k0:k1], vh[k0:k1], scale, p, "bf16", 2.0 ** -8)
        got, gz = o[q0 + at], z[q0 + at]
        none = ~seen.any(1)
        assert np.all(got[none] == 0) and np.all(np.isneginf(gz[none]))
        assert np.all(np.abs(got - want) <= tol), (b, np.abs(got - want).max())
        ok = ~none
        ltol = e + 2.0 ** -22 * np.abs(lw[ok]) + 2.0 ** -20 + 2.0 ** -24 * l
        assert np.all(np.abs(gz[ok] - lw[ok]) <= ltol)


@pytest.mark.parametrize("d,Hq,Hkv,lens,extra", [
    (128, 2, 1, [1], [0]),
    (128, 4, 2, [127, 128, 129, 0, 1, 255, 257], [0] * 7),
    (64, 8, 2, [300, 77, 1, 513], [0] * 4),
    (128, 3, 1, [100, 200, 64], [28, 1000, 128]),           # chunks that end longer prompts
    (64, 5, 5, [256, 5, 31], [1, 123, 0]),
    (128, 2, 2, [200, 130, 300, 40], [-100, -130, -172, -1]),  # queries before the first key
    (128, 8, 1, [700], [0]),
])
def test_ragged_prompts(d, Hq, Hkv, lens, extra):
    M = lib()
    rng = np.random.default_rng(d + sum(lens))
    cu_q, cu_k = cum(lens), cum([a + b for a, b in zip(lens, extra)])
    q = cuda(rng.standard_normal((cu_q[-1], Hq, d)).astype(np.float32) * 2, torch.bfloat16)
    k, v = (cuda(rng.standard_normal((cu_k[-1], Hkv, d)).astype(np.float32), torch.bfloat16) for _ in range(2))
    out, lse = M.misa_prompt_attention(q, k, v, cuda(cu_q), cuda(cu_k), want_lse=True)
    check(M, q, k, v, cu_q, cu_k, out, lse, d ** -0.5)
    M.misa_device_check()


@pytest.mark.parametrize("d", [64, 128])
def test_longer_prompts(d):
    M = lib()
    rng = np.random.default_rng(d)
    lens, extra = [2500, 1700], [0, 3001]
    cu_q, cu_k = cum(lens), cum([a + b for a, b in zip(lens, extra)])
    q = cuda(rng.standard_normal((cu_q[-1], 4, d)).astype(np.float32) * 3, torch.bfloat16)
    k, v = (cuda(rng.standard_normal((cu_k[-1], 2, d)).astype(np.float32), torch.bfloat16) for _ in range(2))
    out, lse = M.misa_prompt_attention(q, k, v, cuda(cu_q), cuda(cu_k), want_lse=True)
    check(M, q, k, v, cu_q, cu_k, out, lse, d ** -0.5, rows=60)
    again, _ = M.misa_prompt_attention(q, k, v, cuda(cu_q), cuda(cu_k))
    assert torch.equal(out, again)
    M.misa_device_check()


@pytest.mark.parametrize("d,Hq,Hkv,lens,extra", [
    (128, 4, 2, [130], [20000]),                     # two items a head, cut between all CTAs
    (64, 2, 1, [1], [9000]),
    (128, 1, 1, [300, 1, 257], [5000, 0, -200]),     # items of every length, some queries before the first key
    (64, 24, 8, [400, 0, 90, 1, 700, 256, 33] * 3, [0] * 21),   # more items than are cut
    (128, 16, 2, [64] * 60 + [900], [0] * 60 + [3000]),
])
def test_items_cut_between_ctas(d, Hq, Hkv, lens, extra):
    M = lib()
    rng = np.random.default_rng(d + len(lens))
    cu_q, cu_k = cum(lens), cum([a + b for a, b in zip(lens, extra)])
    q = cuda(rng.standard_normal((cu_q[-1], Hq, d)).astype(np.float32) * 2, torch.bfloat16)
    k, v = (cuda(rng.standard_normal((cu_k[-1], Hkv, d)).astype(np.float32), torch.bfloat16) for _ in range(2))
    out, lse = M.misa_prompt_attention(q, k, v, cuda(cu_q), cuda(cu_k), want_lse=True)
    check(M, q, k, v, cu_q, cu_k, out, lse, d ** -0.5, rows=12)
    again, al = M.misa_prompt_attention(q, k, v, cuda(cu_q), cuda(cu_k), want_lse=True)
    assert torch.equal(out, again) and torch.equal(lse, al)
    M.misa_device_check()


def test_many_long_items_and_an_output_between_sectors():
    M = lib()
    rng = np.random.default_rng(31)
    lens, extra, Hq, Hkv, d = [1100, 1500, 0, 1300, 1, 900], [0, 0, 0, 1000, 4000, 300], 40, 8, 64
    cu_q, cu_k = cum(lens), cum([a + b for a, b in zip(lens, extra)])
    q = cuda(rng.standard_normal((cu_q[-1], Hq, d)).astype(np.float32) * 2, torch.bfloat16)
    k, v = (cuda(rng.standard_normal((cu_k[-1], Hkv, d)).astype(np.float32), torch.bfloat16) for _ in range(2))
    out, lse = M.misa_prompt_attention(q, k, v, cuda(cu_q), cuda(cu_k), want_lse=True)
    check(M, q, k, v, cu_q, cu_k, out, lse, d ** -0.5, rows=12)
    room = torch.full((q.numel() + 16,), 7.0, dtype=torch.bfloat16, device="cuda")
    other = room[8:8 + q.numel()].view_as(q)  # 16 bytes past a 256-byte boundary
    M.misa_prompt_attention(q, k, v, cuda(cu_q), cuda(cu_k), out=other)
    assert torch.equal(other, out) and (room[:8] == 7).all() and (room[-8:] == 7).all()
    M.misa_device_check()


def test_sharp_and_flat_logits_and_growing_maxima():
    M = lib()
    rng = np.random.default_rng(5)
    cu = cum([600])
    for spread, ramp in ((40.0, False), (1e-3, False), (1.0, True)):
        x = rng.standard_normal((600, 2, 128)).astype(np.float32)
        if ramp:  # keys whose logits keep rising along the prompt, so that the maximum does in every tile
            x = np.abs(x) * np.linspace(0.1, 6, 600, dtype=np.float32)[:, None, None]
        k = cuda(x, torch.bfloat16)
        q = cuda((np.abs(rng.standard_normal((600, 4, 128))) if ramp else rng.standard_normal((600, 4, 128))).astype(np.float32) * spread, torch.bfloat16)
        v = cuda(rng.standard_normal((600, 2, 128)).astype(np.float32), torch.bfloat16)
        out, lse = M.misa_prompt_attention(q, k, v, cuda(cu), want_lse=True, scale=0.07)
        check(M, q, k, v, cu, cu, out, lse, 0.07)


def test_views_of_a_fused_projection_and_rows_of_no_sequence():
    M = lib()
    rng = np.random.default_rng(6)
    Hq, Hkv, d, rows = 6, 2, 64, 450
    fused = cuda(rng.standard_normal((rows, (Hq + 2 * Hkv) * d)).astype(np.float32), torch.bfloat16)
    q = fused[:, :Hq * d].unflatten(1, (Hq, d))
    k = fused[:, Hq * d:(Hq + Hkv) * d].unflatten(1, (Hkv, d))
    v = fused[:, (Hq + Hkv) * d:].unflatten(1, (Hkv, d))
    cu = np.array([10, 140, 140, 401], np.int32)
    out = torch.full((rows, Hq, d), 5.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((rows, Hq), 5.0, device="cuda")
    M.misa_prompt_attention(q, k, v, cuda(cu), out=out, lse=lse)
    check(M, q, k, v, cu, cu, out, lse, d ** -0.5)
    for x in (out, lse):
        assert (x[:10] == 5).all() and (x[401:] == 5).all()


def test_more_sequences_than_threads():
    M = lib()
    rng = np.random.default_rng(16)
    lens = rng.integers(0, 5, 1100)
    cu = cum(lens)
    q = cuda(rng.standard_normal((cu[-1], 2, 64)).astype(np.float32), torch.bfloat16)
    k, v = (cuda(rng.standard_normal((cu[-1], 1, 64)).astype(np.float32), torch.bfloat16) for _ in range(2))
    out, lse = M.misa_prompt_attention(q, k, v, cuda(cu), want_lse=True)
    check(M, q, k, v, cu, cu, out, lse, 0.125)


@pytest.mark.parametrize("junk", [float("nan"), float("inf"), -float("inf")])
def test_rows_of_other_sequences_do_not_reach_a_sequence(junk):
    """Keys and values next to a sequence that are not finite change nothing in it."""
    M = lib()
    rng = np.random.default_rng(7)
    lens = [70, 190, 33, 129]
    cu = cum(lens)
    q = cuda(rng.standard_normal((cu[-1], 4, 128)).astype(np.float32), torch.bfloat16)
    k, v = (cuda(rng.standard_normal((cu[-1], 2, 128)).astype(np.float32), torch.bfloat16) for _ in range(2))
    good, gl = M.misa_prompt_attention(q, k, v, cuda(cu), want_lse=True)
    for b in (0, 2):
        for x in (k, v):
            x[cu[b]:cu[b + 1]] = junk
    bad, bl = M.misa_prompt_attention(q, k, v, cuda(cu), want_lse=True)
    for b in (1, 3):
        assert torch.equal(bad[cu[b]:cu[b + 1]], good[cu[b]:cu[b + 1]])
        assert torch.equal(bl[cu[b]:cu[b + 1]], gl[cu[b]:cu[b + 1]])


@pytest.mark.parametrize("junk", [float("nan"), float("inf")])
def test_tokens_behind_a_query_do_not_reach_it(junk):
    """A key and value that are not finite change no earlier token's output."""
    M = lib()
    rng = np.random.default_rng(8)
    for n, at, Hq in ((300, 150, 4), (300, 290, 4), (1000, 513, 4), (1000, 513, 64), (5000, 4444, 4)):
        cu = cum([n])
        q = cuda(rng.standard_normal((n, Hq, 64)).astype(np.float32), torch.bfloat16)
        k, v = (cuda(rng.standard_normal((n, 2, 64)).astype(np.float32), torch.bfloat16) for _ in range(2))
        good, gl = M.misa_prompt_attention(q, k, v, cuda(cu), want_lse=True)
        k[at], v[at, 0] = junk, junk
        bad, bl = M.misa_prompt_attention(q, k, v, cuda(cu), want_lse=True)
        assert torch.equal(bad[:at], good[:at]) and torch.equal(bl[:at], gl[:at])
        assert not torch.isfinite(bad[at, 0].float()).any()


def test_captured_call_follows_its_inputs():
    M = lib()
    rng = np.random.default_rng(9)
    q = cuda(rng.standard_normal((500, 4, 128)).astype(np.float32), torch.bfloat16)
    k, v = (cuda(rng.standard_normal((500, 2, 128)).astype(np.float32), torch.bfloat16) for _ in range(2))
    cu = cuda(np.array([0, 200, 500], np.int32))
    out, lse = torch.zeros_like(q), torch.zeros(500, 4, device="cuda")
    M.misa_prompt_attention(q, k, v, cu, out=out, lse=lse)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        M.misa_prompt_attention(q, k, v, cu, out=out, lse=lse)
    cu.copy_(cuda(np.array([0, 333, 490], np.int32)))
    q.neg_()
    out.fill_(3)
    g.replay()
    torch.cuda.synchronize()
    want, wl = M.misa_prompt_attention(q, k, v, cu, want_lse=True)
    assert torch.equal(out[:490], want[:490]) and torch.equal(lse[:490], wl[:490]) and (out[490:] == 3).all()
