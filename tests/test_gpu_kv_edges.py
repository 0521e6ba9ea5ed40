"""GPU tests of the plain cache at the ends of what its header promises.
"""
import numpy as np
import pytest
import torch

from rank_quantized_kv_decode_b200 import _lib as L
from test_gpu_kv import Case, f64, near16, rotated

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["bf16", "f16", "int8"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n", [7, 32, 33, 500])  # one launch up to 32 tokens, two beyond
@pytest.mark.parametrize("in_place", [False, True])
def test_queries_of_tokens_outside_the_table_become_zeros_whatever_they_hold(fmt, d, n, in_place):
    c = Case(fmt, 10, 2, d, [64 * 8], width=8, seed=n)
    pos = np.arange(n)
    bad = np.arange(n) % 7 != 3
    pos[bad] = np.resize([-1, 512, 2**31 - 1, -2**31, -64, 513], bad.sum())
    q, k = c.draw(n, 10), c.draw(n, 2)
    # padding of a batch is often not initialised
    rows = torch.from_numpy(np.flatnonzero(bad)).cuda()
    for ch, x in ((0, float("inf")), (5, float("nan")), (d // 2, -float("inf")), (d - 1, float("nan"))):
        q[rows, :, ch] = x
        k[rows, :, ch] = x
    want, tol = rotated(q[~torch.from_numpy(bad)], pos[~bad])
    q_out = q if in_place else torch.full_like(q, 7.0)
    before = c.pages().copy()
    c.append(k, k, np.zeros(n), pos, q=q, q_out=q_out)
    assert c.status() == L.DEV_BOUNDS
    near16(f64(q_out)[~bad], want, tol, fmt)
    assert not q_out[rows].view(torch.int16).any()
    # the pages changed at the good tokens' alone
    page = c.table_np[0][pos[~bad] // 64]
    others = np.setdiff1d(np.arange(before.shape[0]), page)
    assert np.array_equal(before[others], c.pages()[others])
