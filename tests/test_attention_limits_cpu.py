"""Refusals and sizes of the attention calls at the edges of what they serve, on a machine without a GPU."""
import ctypes

import pytest

from long_context_sparse_mean_b200 import build

OK, INVALID = 0, 1
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
