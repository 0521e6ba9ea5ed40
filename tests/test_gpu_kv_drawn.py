"""GPU parity of the plain cache's decode where its list of tiles is long enough that the warps draw the
end of it: few CTAs make that of a few thousand tiles.  Tolerances are those of test_gpu_kv.py, whose
sums do not depend on the number of chunks.
"""
import numpy as np
import pytest
import torch

from rank_quantized_kv_decode_b200 import api
from test_gpu_kv import Case

pytestmark = pytest.mark.gpu

WARPS = 4      # of a CTA of the split kernel
DRAWN_AT = 40  # tiles a warp above which some are drawn
TILE = {"bf16": 16, "f16": 16, "int8": 32}


def draws(c, ctas, pages=None):
    """Whether a call over ``pages`` pages of each sequence (default: all) draws."""
    groups = -(-c.H // c.Hkv // 8)
    pages = [-(-n // 64) for n in c.lens] if pages is None else pages
    return sum(pages) * c.Hkv * groups * (64 // TILE[c.fmt]) > ctas * WARPS * DRAWN_AT


@pytest.mark.parametrize("fmt", ["bf16", "f16", "int8"])
@pytest.mark.parametrize("H,Hkv,d,ctas", [(8, 2, 128, 1), (8, 2, 128, 4), (6, 2, 64, 1), (6, 2, 64, 3), (20, 2, 64, 7),
                                          (32, 2, 128, 8)])
def test_drawn_chunks_match_the_oracle_and_repeat(fmt, H, Hkv, d, ctas):
    c = Case(fmt, H, Hkv, d, [1500, 17, 0, 9000, 640, 1], seed=H + d + ctas)
    assert draws(c, ctas)
    c.fill()
    q = c.draw(6, H, 1.5)
    out, lse = c.decode(q, max_ctas=ctas)
    assert c.status() == 0
    c.check(q, out, lse)
    for _ in range(3):
        again, lse2 = c.decode(q, max_ctas=ctas)
        assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("fmt,lens", [("bf16", [40 * i for i in range(70)]), ("int8", [64] * 33 + [0, 5000, 1]),
                                      ("f16", [0] * 31 + [7000] + [0] * 31 + [1])])
def test_drawn_chunks_of_batches_beyond_a_warp(fmt, lens):
    c = Case(fmt, 2, 2, 64, lens, seed=len(lens))
    assert draws(c, 1)
    c.fill()
    q = c.draw(len(lens), 2, 1.5)
    out, lse = c.decode(q, max_ctas=1)
    assert c.status() == 0
    c.check(q, out, lse)


@pytest.mark.parametrize("fmt", ["bf16", "f16", "int8"])
def test_drawn_chunks_of_a_window_and_of_a_selection(fmt):
    c = Case(fmt, 8, 2, 128, [300, 9000, 64 * 50], seed=17)
    c.fill()
    q = c.draw(3, 8, 1.5)
    assert draws(c, 1, [5, 65, 50])
    out, lse = c.decode(q, window=4100, max_ctas=1)
    c.check(q, out, lse, window=4100)
    sel = np.full((3, 2, 60), -1, np.int32)
    for b, n in enumerate(c.lens):
        P = -(-n // 64)
        for g in range(2):
            m = min(P, 60)
            sel[b, g, :m] = np.sort(c.rng.choice(P, m, replace=False))
    assert draws(c, 1, [5, 60, 50])
    out, lse = c.decode(q, sel=torch.from_numpy(sel).cuda(), max_ctas=1)
    assert c.status() == 0
    c.check(q, out, lse, sel=sel)


@pytest.mark.parametrize("fmt", ["bf16", "int8"])
def test_drawing_calls_may_find_anything_in_the_workspace(fmt):
    """Zeros, ones, noise, what a call of other sizes left: the same bits."""
    c = Case(fmt, 8, 2, 128, [3000, 17, 9000, 640], seed=13)
    o = Case("f16", 4, 4, 64, [5000, 100], seed=14)
    assert draws(c, 2) and draws(o, 1)
    c.fill()
    o.fill()
    q, qo = c.draw(4, 8, 1.5), o.draw(2, 4)
    out, lse = c.decode(q, max_ctas=2)
    c.check(q, out, lse)
    want = o.decode(qo, max_ctas=1)
    o.check(qo, *want)
    ws = o.kv.decode_ws = c.kv.decode_ws
    g = torch.Generator("cuda").manual_seed(5)
    for fill in (0x00, 0xFF, 0x80, None):
        if fill is None:
            ws.copy_(torch.randint(0, 256, ws.shape, dtype=torch.uint8, device="cuda", generator=g))
        else:
            ws.fill_(fill)
        for _ in range(3):
            again, lse2 = c.decode(q, max_ctas=2)
            assert torch.equal(out, again) and torch.equal(lse, lse2), fill
            other = o.decode(qo, max_ctas=1)
            assert all(torch.equal(x, y) for x, y in zip(want, other)), fill


@pytest.mark.parametrize("fmt", ["bf16", "f16", "int8"])
@pytest.mark.parametrize("upper", [0, 1, 0x73744B56])
def test_a_count_left_in_the_workspace_skips_nothing(fmt, upper):
    """The first words of a workspace as a call that did not finish might leave them, beside records that
    are none of this call's."""
    c = Case(fmt, 8, 2, 128, [3000, 17, 9000, 640], seed=13)
    assert draws(c, 2)
    c.fill()
    q = c.draw(4, 8, 1.5)
    out, lse = c.decode(q, max_ctas=2)
    c.check(q, out, lse)
    ws = c.kv.decode_ws
    for count in (1, 7, 20, 1 << 20, 0x73744B56, 0xFFFFFFFF):
        ws.fill_(0xFF)
        word = torch.tensor(np.array([upper << 32 | count], np.uint64).view(np.int64))
        ws[:8].view(torch.int64).copy_(word)
        again, lse2 = c.decode(q, max_ctas=2)
        assert torch.equal(out, again) and torch.equal(lse, lse2), count
        again, lse2 = c.decode(q, max_ctas=2)
        assert torch.equal(out, again) and torch.equal(lse, lse2), count
    assert c.status() == 0


def test_a_captured_call_draws_at_some_lengths_and_not_at_others():
    c = Case("bf16", 8, 2, 128, [5000, 900, 64], seed=3)
    c.fill()
    full = list(c.lens)
    q = c.draw(3, 8, 1.5)
    out = torch.empty_like(q)
    lse = torch.empty(3, 8, device="cuda")

    def step():
        api.kv_decode(c.lay, q, c.kv.cache, c.table, c.len_t, out, c.kv.decode_ws, c.kv.status, lse=lse, max_ctas=2)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for lens, many in ((full, True), ([130, 900, 64], False), ([4000, 1, 0], True), ([0, 0, 0], False), (full, True)):
        c.lens = lens
        assert draws(c, 2) == many
        c.len_t.copy_(torch.tensor(lens))
        graph.replay()
        c.check(q, out, lse)
        first = out.clone()
        graph.replay()
        assert torch.equal(first, out)
        eager, _ = c.decode(q, max_ctas=2)
        assert torch.equal(eager, out)
    assert c.status() == 0


def test_two_streams_that_draw_from_a_workspace_each():
    cs = [Case("bf16", 8, 2, 128, [6000 - 700 * i, 5000], seed=i) for i in range(2)]
    for c in cs:
        assert draws(c, 2)
        c.fill()
    qs = [c.draw(2, 8, 1.5) for c in cs]
    streams = [torch.cuda.Stream() for _ in cs]
    outs = [(torch.empty_like(q), torch.empty(2, 8, device="cuda")) for q in qs]
    torch.cuda.synchronize()
    for _ in range(20):
        for c, q, (o, l), st in zip(cs, qs, outs, streams):
            api.kv_decode(c.lay, q, c.kv.cache, c.table, c.len_t, o, c.kv.decode_ws, c.kv.status, lse=l, max_ctas=2,
                          stream=st)
    torch.cuda.synchronize()
    for c, q, (o, l) in zip(cs, qs, outs):
        c.check(q, o, l)
