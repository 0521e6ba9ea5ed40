"""GPU tests of the plain cache at the ends of what its header promises.
"""
import numpy as np
import pytest
import torch

from oracle import kv_oracle as K
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


@pytest.mark.parametrize("width", [9, 200])  # one CTA a choice, and several
@pytest.mark.parametrize("n,n_sel,first,last,bad", [
    (64 * 5, 8, 1, 2, 3), (64 * 5, 5, 0, 1, 0), (1, 1, 0, 1, 0), (64 * 5 - 7, 5, 1, 1, 4),  # every page is taken
    (64 * 9, 3, 1, 2, 0), (64 * 9, 3, 1, 2, 7), (64 * 9, 2, 0, 2, 8), (64 * 9, 3, 1, 2, 4),  # none is scored
    (64 * 9, 6, 2, 3, 1), (64 * 9, 6, 2, 3, 6), (64 * 9, 6, 2, 3, 8), (64 * 9 - 63, 5, 1, 1, 8),  # kept at an end
    (64 * 9, 6, 2, 3, 4)])  # scored
def test_select_flags_a_bad_page_wherever_it_lies(width, n, n_sel, first, last, bad):
    c = Case("bf16", 4, 2, 64, [64 * 9, n], seed=2, width=width)
    c.fill()
    q = c.draw(2, 4)
    s = K.page_scores(f64(q)[1], K.read_bounds(c.pages(), c.olay)[c.table_np[1, :-(-n // 64)]])
    c.table[1, -(-n // 64):] = -1  # behind the sequence: no entries of its own
    c.select(q, n_sel, first, last)
    assert c.status() == 0
    for entry in (-1, c.kv.num_pages, 2**31 - 1, -2**31):
        c.kv.status.zero_()
        c.table[1, bad] = entry
        sel = c.select(q, n_sel, first, last).cpu().numpy()
        assert c.status() == L.DEV_BOUNDS, entry
        s[:, bad] = -np.inf
        for g in range(2):
            assert np.array_equal(sel[1, g], K.choose(s[g], n, n_sel, first, last))


@pytest.mark.parametrize("d,H", [(64, 1), (128, 2), (64, 10)])
@pytest.mark.parametrize("power", [-149, -144, -140, -130, -120, -110, 0, 110, 119, 120, 121, 122, 123, 124])
def test_select_at_the_ends_of_fp32(power, d, H):
    """Bounds above zero under queries of both signs: a score is the difference of two sums of about 2^power times the
    number of channels, which pass fp32's largest number, or fall below its smallest, where the score is exact."""
    pages = 300
    c = Case("bf16", H, 1, d, [64 * pages], seed=200 + d + power, fill=0)
    x = 1.0 + np.abs(c.rng.standard_normal((c.kv.num_pages, 2, d)))
    x[:, 1] = x[:, 0] * (1 + 0.2 * c.rng.random(x[:, 0].shape))
    bits = torch.from_numpy(x * 2.0 ** (power // 2)).bfloat16().view(torch.int16).numpy()
    img = c.pages().copy()
    img[:, :c.olay["off_heads"]] = bits.reshape(c.kv.num_pages, -1).view(np.uint8)
    c.kv.cache.copy_(torch.from_numpy(img.reshape(-1)))
    q = c.draw(1, H, 2.0 ** (power - power // 2))
    s = K.page_scores(f64(q)[0], K.read_bounds(img, c.olay)[c.table_np[0]])
    assert np.all(np.isfinite(s)) and len(np.unique(s)) > pages - 3
    for n_sel in (3, 20, 150, 298):
        sel = c.select(q, n_sel, 1, 1).cpu().numpy()
        assert np.array_equal(sel[0, 0], K.choose(s[0], 64 * pages, n_sel, 1, 1)), n_sel
    assert c.status() == 0
