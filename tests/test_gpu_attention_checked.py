"""The bounds-checked build counts what the attention calls skip: page-table entries outside the pool and token
ids outside the prefix.  A child process loads the checked library; the ids are ones every build skips."""
import json
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)


def _child():
    import torch

    from long_context_sparse_mean_b200 import build
    build.build(checked=True)
    from long_context_sparse_mean_b200 import binding as M
    assert M.checked_build()
    M.misa_bad_index_counts()
    T, Hq, Hkv, d, page, per = 2, 24, 2, 128, 64, 8
    cap = per * page
    gen = torch.Generator("cuda").manual_seed(1)
    rand = lambda *s: torch.randn(*s, device="cuda", generator=gen).bfloat16()  # noqa: E731
    ints = lambda x: torch.tensor(x, device="cuda", dtype=torch.int32)  # noqa: E731
    pool = M.misa_kv4_pool(T * per, page, Hkv, d)
    good = torch.arange(T * per, device="cuda", dtype=torch.int32).reshape(T, per)
    table = good.clone()
    table[1, 3] = T * per
    k, v, q = rand(T * cap, Hkv, d), rand(T * cap, Hkv, d), rand(T, Hq, d)
    cu, zero, n = ints([0, cap, 2 * cap]), ints([0, 0]), ints([cap, cap - 7])
    out = {}

    def count(name, call):
        call()
        out[name] = M.misa_bad_index_counts()

    idx = torch.full((T, 40), -1, device="cuda", dtype=torch.int32)
    idx[:, 3:20] = torch.arange(17, device="cuda", dtype=torch.int32) * 11
    count("clean append", lambda: M.misa_kv4_append(k, v, pool, good, cu, zero))
    count("clean attention", lambda: M.misa_kv4_attention(q, pool, good, n, idx=idx))
    idx[0, 30], idx[1, 31], idx[1, 32] = -7, cap - 7, 1 << 30
    count("append", lambda: M.misa_kv4_append(k, v, pool, table, cu, zero))
    count("read", lambda: M.misa_kv4_read(pool, table, cu, zero, T * cap, d))
    count("whole", lambda: M.misa_kv4_attention(q, pool, table, n))
    count("selected", lambda: M.misa_kv4_attention(q, pool, good, n, idx=idx))
    keep = torch.arange(100, 300, device="cuda", dtype=torch.int32).expand(T, -1).contiguous()
    count("close up", lambda: M.misa_kv4_compact(pool, table, keep, d))
    print(json.dumps(out))


def test_checked_build_counts_what_attention_skips():
    env = dict(os.environ, MISA_LIBRARY="checked")
    code = ("import sys; sys.path[:0] = [%r, %r]; import test_gpu_attention_checked as t; t._child()" % (ROOT, HERE))
    r = subprocess.run([sys.executable, "-c", code], env=env, capture_output=True, text=True, timeout=900, cwd=ROOT)
    assert r.returncode == 0, r.stderr[-3000:]
    assert json.loads(r.stdout.strip().splitlines()[-1]) == {
        "clean append": [0, 0, 0], "clean attention": [0, 0, 0],
        "append": [0, 0, 64], "read": [0, 0, 64],       # a page of 64 rows
        "whole": [0, 0, 4],                             # looked up for 16 rows at a time
        "selected": [0, 3, 0],
        "close up": [0, 0, 64],                         # rows 192 .. 255 are sources
    }
