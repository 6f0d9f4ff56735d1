"""Refusals of the attention calls on a machine without a GPU: every bad argument is rejected on the host,
by the C library before any launch and by the binding before any device check."""
import ctypes

import pytest
import torch

from long_context_sparse_mean_b200 import build

OK, INVALID, UNSUPPORTED, WORKSPACE = range(4)
BF16, F32 = 0, 1
P = ctypes.c_void_p
FAKE, BENT = P(0x10000), P(0x10008)  # never dereferenced: every call below fails validation first
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def M():
    build.build()
    from long_context_sparse_mean_b200 import binding
    return binding


@pytest.fixture(scope="module")
def lib(M):
    return M.library()


def call(fn, base, **kw):
    assert not set(kw) - set(base), set(kw) - set(base)
    return fn(*{**base, **kw}.values())


APPEND = dict(k=FAKE, v=FAKE, ldk=1024, ldv=1024, dt=BF16, kg=1.0, vg=1.0, pool=FAKE, np=100, ps=64, table=FAKE, mp=10,
              cu=FAKE, start=FAKE, S=2, rows=8, H=8, d=128, s=None)
READ = dict(pool=FAKE, np=100, ps=64, table=FAKE, mp=10, cu=FAKE, start=FAKE, S=2, rows=8, H=8, d=128, dt=BF16, kg=1.0,
            vg=1.0, k=FAKE, v=FAKE, s=None)
ATTEND = dict(q=FAKE, pool=FAKE, np=100, ps=64, table=FAKE, mp=10, n=FAKE, idx=None, T=4, L=640, P=0, Hq=32, H=8, d=128,
              dt=BF16, scale=0.1, kg=1.0, vg=1.0, out=FAKE, lse=None, acc=None, ld=0, ws=FAKE, wsb=1 << 30, s=None)
EVICT = dict(acc=FAKE, ld=1000, n=FAKE, T=4, L=1000, keep=100, sink=4, recent=20, idx=FAKE, no=FAKE, out=None, ldo=0,
             s=None)
COMPACT = dict(pool=FAKE, np=100, ps=64, table=FAKE, mp=10, idx=FAKE, T=4, keep=100, H=8, d=128, ws=FAKE, wsb=1 << 30,
               s=None)
KEYS = dict(pool=FAKE, np=100, ps=64, table=FAKE, mp=10, idx=FAKE, T=4, keep=100, d=128, dt=BF16, ws=FAKE, wsb=1 << 30,
            s=None)
PROMPT = dict(q=FAKE, k=FAKE, v=FAKE, ldq=4096, ldk=1024, ldv=1024, cuq=FAKE, cuk=FAKE, S=2, Tq=8, Tk=8, Hq=32, H=8,
              d=128, dt=BF16, scale=0.1, out=FAKE, lse=None, ws=FAKE, wsb=1 << 30, s=None)


@pytest.mark.parametrize("name,base", [("misa_kv4_append", APPEND), ("misa_kv4_read", READ)])
def test_cache_refusals(lib, name, base):
    fn = getattr(lib, name)
    for kw, want in [(dict(d=96), UNSUPPORTED), (dict(ps=60), UNSUPPORTED), (dict(ps=1040), UNSUPPORTED),
                     (dict(dt=3), UNSUPPORTED), (dict(np=1 << 40), UNSUPPORTED), (dict(H=0), INVALID),
                     (dict(S=-1), INVALID), (dict(rows=-1), INVALID), (dict(np=0), INVALID), (dict(mp=0), INVALID),
                     (dict(kg=0.0), INVALID), (dict(vg=-1.0), INVALID), (dict(kg=NAN), INVALID), (dict(vg=INF), INVALID),
                     (dict(kg=2.0 ** -61), INVALID), (dict(vg=2.0 ** 61), INVALID),
                     (dict(pool=None), INVALID), (dict(pool=BENT), INVALID), (dict(table=None), INVALID),
                     (dict(cu=None), INVALID), (dict(start=None), INVALID), (dict(k=None), INVALID),
                     (dict(v=BENT), INVALID), (dict(rows=1 << 30), UNSUPPORTED),
                     (dict(rows=0, k=None, v=None, pool=None), OK), (dict(S=0, cu=None, start=None), OK)]:
        assert call(fn, base, **kw) == want, kw
    if name == "misa_kv4_append":
        for kw in (dict(ldk=1023), dict(ldv=1028), dict(ldk=1000)):
            assert call(fn, base, **kw) == INVALID, kw


def test_attention_refusals(lib):
    fn = lib.misa_kv4_attention
    for kw, want in [(dict(d=32), UNSUPPORTED), (dict(ps=24), UNSUPPORTED), (dict(dt=2), UNSUPPORTED),
                     (dict(Hq=30), INVALID), (dict(Hq=0), INVALID), (dict(L=0), INVALID), (dict(L=641), INVALID),
                     (dict(T=-1), INVALID), (dict(idx=FAKE, P=0), INVALID), (dict(scale=0.0), INVALID),
                     (dict(scale=NAN), INVALID), (dict(kg=-1.0), INVALID), (dict(acc=FAKE, ld=639), INVALID),
                     (dict(q=None), INVALID), (dict(q=BENT), INVALID), (dict(out=None), INVALID), (dict(n=None), INVALID),
                     (dict(out=BENT), INVALID), (dict(ws=None), WORKSPACE), (dict(ws=BENT), WORKSPACE),
                     (dict(wsb=100), WORKSPACE), (dict(acc=FAKE, ld=640, wsb=lib.misa_workspace_bytes(11, 4, 640, 32, 8, 128, 0, 0)), WORKSPACE),
                     (dict(T=0, q=None, out=None, n=None, ws=None), OK)]:
        assert call(fn, ATTEND, **kw) == want, kw


def test_eviction_refusals(lib):
    for kw, want in [(dict(keep=0), INVALID), (dict(sink=-1), INVALID), (dict(sink=81), INVALID), (dict(ld=999), INVALID),
                     (dict(sink=1 << 30, recent=(1 << 31) - 1), INVALID), (dict(T=-1), INVALID), (dict(L=0), INVALID),
                     (dict(idx=None), INVALID), (dict(no=None), INVALID), (dict(acc=None), INVALID),
                     (dict(out=FAKE, ldo=1000), INVALID),  # the kept weights over the ones still read
                     (dict(out=P(0x10000 + 4 * 3999), ldo=100), INVALID), (dict(out=P(1 << 30), ldo=99), INVALID),
                     (dict(T=0, acc=None, idx=None), OK)]:
        assert call(lib.misa_evict_select, EVICT, **kw) == want, kw
    for kw, want in [(dict(keep=0), INVALID), (dict(keep=641), INVALID), (dict(d=100), UNSUPPORTED), (dict(ps=8), UNSUPPORTED),
                     (dict(idx=None), INVALID), (dict(pool=BENT), INVALID), (dict(ws=None), WORKSPACE),
                     (dict(ws=BENT), WORKSPACE), (dict(wsb=4), WORKSPACE), (dict(T=0, idx=None), OK)]:
        assert call(lib.misa_kv4_compact, COMPACT, **kw) == want, kw
    for kw, want in [(dict(keep=0), INVALID), (dict(keep=641), INVALID), (dict(d=64), UNSUPPORTED), (dict(dt=5), UNSUPPORTED),
                     (dict(idx=None), INVALID), (dict(pool=BENT), INVALID), (dict(ws=None), WORKSPACE),
                     (dict(ws=BENT), WORKSPACE), (dict(wsb=4), WORKSPACE), (dict(T=0, idx=None), OK)]:
        assert call(lib.misa_keys_compact_paged, KEYS, **kw) == want, kw


def test_prompt_refusals(lib):
    for kw, want in [(dict(dt=F32), UNSUPPORTED), (dict(d=80), UNSUPPORTED), (dict(Hq=12), INVALID), (dict(Hq=0), INVALID),
                     (dict(H=0), INVALID), (dict(S=-1), INVALID), (dict(Tq=-1), INVALID), (dict(Tk=-1), INVALID),
                     (dict(scale=-0.1), INVALID), (dict(scale=INF), INVALID), (dict(q=None), INVALID), (dict(k=BENT), INVALID),
                     (dict(ldq=4092), INVALID), (dict(ldk=1016), INVALID), (dict(ldv=1027), INVALID), (dict(out=None), INVALID),
                     (dict(out=BENT), INVALID), (dict(cuq=None), INVALID), (dict(cuk=None), INVALID),
                     (dict(Tk=9000, ws=None), WORKSPACE), (dict(Tk=9000, ws=BENT), WORKSPACE), (dict(Tk=9000, wsb=1000), WORKSPACE),
                     (dict(Tq=0, q=None, out=None), OK), (dict(S=0, cuq=None), OK)]:
        assert call(lib.misa_prompt_attention, PROMPT, **kw) == want, kw


def test_workspace_sizes(lib):
    ws = lib.misa_workspace_bytes
    assert ws(11, 0, 100, 32, 8, 128, 0, 0) == 0 and ws(11, 4, 100, 30, 8, 128, 0, 0) == 0
    plain, weights = ws(11, 4, 1000, 32, 8, 128, 0, 0), ws(11, 4, 1000, 32, 8, 128, 0, 1)
    assert weights >= plain + 4 * 32 * 1000 * 4  # the logits
    assert ws(11, 4, 1 << 20, 32, 8, 128, 0, 0) == plain  # without weights it does not grow with the length
    assert ws(11, 4, 1 << 20, 32, 8, 128, 64, 1) < weights


def _t(*s, dtype=torch.bfloat16):
    return torch.zeros(s, dtype=dtype)


def test_binding_checks_shapes_before_the_device(M):
    i32, u8, f32 = torch.int32, torch.uint8, torch.float32
    pool, table = _t(5, 2, 2, 16 * 72, dtype=u8), _t(3, 4, dtype=i32)
    cu, start, n = _t(4, dtype=i32), _t(3, dtype=i32), _t(3, dtype=i32)
    q, acc, idx = _t(3, 8, 128), _t(3, 64, dtype=f32), _t(3, 10, dtype=i32)

    def refuses(what, fn):
        with pytest.raises(ValueError, match=what):
            fn()

    dev = "CUDA tensor"
    refuses(dev, lambda: M.misa_kv4_append(_t(9, 2, 128), _t(9, 2, 128), pool, table, cu, start))
    refuses("k must be", lambda: M.misa_kv4_append(_t(9, 256), _t(9, 256), pool, table, cu, start))
    refuses(dev, lambda: M.misa_kv4_read(pool, table, cu, start, 9, 128))
    refuses("k must be", lambda: M.misa_kv4_read(pool, table, cu, start, 9, 128, k=_t(8, 2, 128)))
    refuses("start must be", lambda: M.misa_kv4_read(pool, table, cu, start[:2], 9, 128))
    refuses("page_table must be", lambda: M.misa_kv4_read(pool, table[:2], cu, start, 9, 128))
    refuses("pool must be", lambda: M.misa_kv4_read(pool[..., :100], table, cu, start, 9, 128))
    refuses(dev, lambda: M.misa_kv4_attention(q, pool, table, n, idx=idx, acc=acc))
    refuses("q must be", lambda: M.misa_kv4_attention(q[0], pool, table, n))
    refuses("n must be", lambda: M.misa_kv4_attention(q, pool, table, n[:2]))
    refuses("idx must be", lambda: M.misa_kv4_attention(q, pool, table, n, idx=idx[:2]))
    refuses("acc must be", lambda: M.misa_kv4_attention(q, pool, table, n, acc=acc[:, :60], L=61))
    refuses("out must be", lambda: M.misa_kv4_attention(q, pool, table, n, out=q[:2]))
    refuses("lse must be", lambda: M.misa_kv4_attention(q, pool, table, n, lse=acc))
    refuses(dev, lambda: M.misa_evict_select(acc, n, 10, 2, 3))
    refuses("acc must be", lambda: M.misa_evict_select(acc[0], n, 10))
    refuses("n must be", lambda: M.misa_evict_select(acc, n[:1], 10))
    refuses("idx must be", lambda: M.misa_evict_select(acc, n, 11, idx=idx))
    refuses("acc_out must be", lambda: M.misa_evict_select(acc, n, 11, acc_out=_t(3, 10, dtype=f32)))
    refuses(dev, lambda: M.misa_kv4_compact(pool, table, idx, 128))
    refuses("idx must be", lambda: M.misa_kv4_compact(pool, table, idx[0], 128))
    refuses(dev, lambda: M.misa_keys_compact_paged(_t(5, 16, 128), table, idx))
    refuses("pool must be", lambda: M.misa_keys_compact_paged(_t(5, 16), table, idx))
    refuses(dev, lambda: M.misa_prompt_attention(_t(9, 8, 64), _t(9, 2, 64), _t(9, 2, 64), cu))
    refuses("d of 64 or 128", lambda: M.misa_kv4_pool(4, 64, 2, 96, device="cpu"))
    refuses("d of 64 or 128", lambda: M.misa_kv4_pool(4, 40, 2, 64, device="cpu"))
    assert tuple(M.misa_kv4_pool(4, 48, 2, 64, device="cpu").shape) == (4, 2, 2, 48 * 36)
