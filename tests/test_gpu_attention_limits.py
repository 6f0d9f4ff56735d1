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
