"""Refusals and sizes of the attention calls at the edges of what they serve, on a machine without a GPU."""
import ctypes

import pytest
import torch

from long_context_sparse_mean_b200 import build

OK, INVALID, UNSUPPORTED, WORKSPACE = range(4)
P = ctypes.c_void_p
FAKE = P(0x10000)  # never dereferenced: every call below fails validation first


@pytest.fixture(scope="module")
def M():
    build.build()
    from long_context_sparse_mean_b200 import binding
    return binding


@pytest.fixture(scope="module")
def lib(M):
    return M.library()


def test_eviction_refuses_lengths_that_overlap_their_outputs(lib):
    """A row's new length over another row's old one: which is read or written first is not said."""
    def select(n, n_out, T=4):
        return lib.misa_evict_select(FAKE, 1000, P(n), T, 1000, 100, 4, 20, FAKE, P(n_out), None, 0, None)

    for n_out in (0x20000 + 4, 0x20000 + 12, 0x20000 - 4, 0x20000 - 12):
        assert select(0x20000, n_out) == INVALID, hex(n_out)
    assert select(0x20000, 0x20000, T=0) == OK


def test_workspace_of_widths_that_no_call_serves_is_zero(lib):
    """Sizes are asked for before the call can refuse them: every width, head count and length gets an answer."""
    ws = lib.misa_workspace_bytes
    ATTEND, CLOSE_UP, KEYS, PROMPT = 11, 12, 13, 14
    odd = (-(1 << 31), -64, -1, 0, 1, 2, 7, 8, 15, 16, 31, 32, 48, 63, 65, 72, 96, 127, 129, 192, 1 << 20, (1 << 31) - 1)
    for h in odd + (256, 512):
        assert ws(ATTEND, 4, 1000, 32, 8, h, 0, 1) == 0, h
        assert ws(CLOSE_UP, 4, 0, 8, 0, h, 1000, 0) == 0, h
        assert ws(PROMPT, 3000, 9000, 32, 2, h, 0, 0) == 0, h
    for h in odd + (64, 128):
        assert ws(KEYS, 4, 0, 0, 0, h, 1000, 0) == 0, h
    for h in (64, 128):
        assert ws(ATTEND, 4, 1000, 32, 8, h, 0, 1) > 0 and ws(CLOSE_UP, 4, 0, 8, 0, h, 1000, 0) > 0
        assert ws(PROMPT, 3000, 9000, 32, 2, h, 0, 0) > 0
        for many in (1025, 1 << 30, (1 << 31) - 1):  # heads
            assert ws(CLOSE_UP, 4, 0, many, 0, h, 1000, 0) == 0 and ws(PROMPT, 3000, 9000, many, 2, h, 0, 0) == 0
            assert ws(ATTEND, 4, 1000, many, many, h, 0, 0) == 0
        assert ws(ATTEND, 4, 1000, 1 << 17, 8, h, 0, 0) == 0
    for h in (256, 512):
        assert ws(KEYS, 4, 0, 0, 0, h, 1000, 0) > 0
    for far in ((1 << 30) + 1, (1 << 31) - 1):  # tokens
        assert ws(ATTEND, 4, far, 32, 8, 128, 0, 0) == 0 and ws(ATTEND, 4, 1000, 32, 8, 128, far, 0) == 0
        assert ws(CLOSE_UP, 4, 0, 8, 0, 128, far, 0) == 0 and ws(KEYS, 4, 0, 0, 0, 256, far, 0) == 0
        assert ws(PROMPT, far, 9000, 32, 2, 128, 0, 0) == 0 and ws(PROMPT, 3000, far, 32, 2, 128, 0, 0) == 0


def test_attention_refuses_sums_that_end_before_the_last_page(M, lib):
    """Without L a prefix may be as long as the table reaches, so acc has to reach the table's last page."""
    zeros = lambda *s, dtype=torch.int32: torch.zeros(s, dtype=dtype)  # noqa: E731
    pool, table, n = zeros(12, 2, 2, 16 * 72, dtype=torch.uint8), zeros(3, 4), zeros(3)
    q = zeros(3, 8, 128, dtype=torch.bfloat16)
    for cols, what in ((10, "acc must be"), (48, "acc must be"), (49, "CUDA tensor"), (64, "CUDA tensor"), (99, "CUDA tensor")):
        with pytest.raises(ValueError, match=what):
            M.misa_kv4_attention(q, pool, table, n, acc=zeros(3, cols, dtype=torch.float32))
    for cols, what in ((39, "acc must be"), (40, "CUDA tensor")):
        with pytest.raises(ValueError, match=what):
            M.misa_kv4_attention(q, pool, table, n, acc=zeros(3, cols, dtype=torch.float32), L=40)

    def attend(cols, ld, acc=FAKE, ws=None):
        return lib.misa_kv4_attention_cols(FAKE, FAKE, 100, 64, FAKE, 10, FAKE, None, 4, 640, 0, 32, 8, 128, 0, 0.1, 1.0, 1.0,
                                           FAKE, None, acc, cols, ld, ws, 0, None)

    assert attend(0, 100) == INVALID and attend(-1, 100) == INVALID and attend(101, 100) == INVALID
    assert attend(100, 100) == WORKSPACE and attend(0, 0, acc=None) == WORKSPACE  # nothing to refuse but the scratch


def test_attention_refuses_a_selection_without_columns(M):
    """An empty tensor has no address, which the library takes for 'no selection, the whole prefix'."""
    zeros = lambda *s, dtype=torch.int32: torch.zeros(s, dtype=dtype)  # noqa: E731
    pool, q = zeros(12, 2, 2, 16 * 72, dtype=torch.uint8), zeros(3, 8, 128, dtype=torch.bfloat16)
    assert zeros(3, 0).data_ptr() == 0
    with pytest.raises(ValueError, match="idx must be"):
        M.misa_kv4_attention(q, pool, zeros(3, 4), zeros(3), idx=zeros(3, 0))


def test_workspace_of_closing_up_holds_marks_and_counters(lib):
    """A mark for each segment of rows and a counter for each sequence and group that hands segments out."""
    ws = lib.misa_workspace_bytes
    for T, Hkv, d, keep in ((1, 1, 64, 40), (3, 8, 128, 20000), (16, 8, 128, 8192), (70000, 1, 64, 600)):
        need = ws(12, T, 0, Hkv, 0, d, keep, 0)
        words = 3 if keep > 512 else 2  # a long list is two segments at least
        assert need % 4 == 0 and need >= words * 4 * T, (T, keep)
        keys = ws(13, T, 0, 0, 0, 256, keep, 0)
        assert keys % 4 == 0 and keys >= words * 4 * T


def test_workspace_of_summed_weights_is_bounded(lib):
    """The logits of as many queries as 1 GiB holds, one at least; never more than the call's own."""
    ws = lib.misa_workspace_bytes
    for T, L, Hq, Hkv in ((256, 131072, 64, 8), (4096, 131072, 128, 1), (256, 1 << 20, 8, 8)):
        plain, weights = ws(11, T, L, Hq, Hkv, 128, 0, 0), ws(11, T, L, Hq, Hkv, 128, 0, 1)
        one = 4 * Hq * (L + 128)
        assert max(1 << 29, one) < weights <= plain + max(1 << 30, one) + 4 * 256 * Hq + 4096, (T, L, Hq)
    assert ws(11, 16, 131072, 64, 8, 128, 0, 1) >= 16 * 131072 * 64 * 4  # half a GiB: in one go
    assert ws(11, 1, 1 << 24, 256, 1, 128, 0, 1) >= (1 << 24) * 256 * 4  # a single query always


def test_a_workspace_keeps_the_buffers_that_captured_calls_use(M, monkeypatch):
    """A graph writes to the scratch it was captured with at every replay, also after the workspace has grown."""
    import contextlib
    import gc
    import types
    import weakref

    capturing = [False]
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: types.SimpleNamespace(cuda_stream=7))
    monkeypatch.setattr(torch.cuda, "stream", lambda stream: contextlib.nullcontext())
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: capturing[0])

    def get(ws, nbytes, capture, how):
        capturing[0] = capture
        if how == "get":
            buf = ws.get(nbytes)
        else:
            buf = M._scratch(ws, torch.zeros(1), 0, nbytes, None, 7)
        capturing[0] = False
        return weakref.ref(buf)

    for how in ("get", "scratch"):
        ws = M.Workspace("cpu")
        eager = get(ws, 1 << 10, False, how)
        same = get(ws, 1 << 9, True, how)
        assert same() is eager() is ws.buf
        later = get(ws, 1 << 12, False, how)
        gc.collect()
        assert same() is not None and later() is not same(), how
        grown = get(ws, 1 << 14, True, how)  # nothing captured used the one before
        last = get(ws, 1 << 16, False, how)
        gc.collect()
        assert later() is None and grown() is not None and same() is not None and last() is ws.buf, how
        ws.release()
        gc.collect()
        assert same() is None and grown() is None and last() is None and ws.buf is None
