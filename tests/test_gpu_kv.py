"""GPU parity of the plain key-value cache with the fp64 oracle: append (rotation, storage, bounds),
read-back, decode attention, choice of pages, attention over a choice, and the run of them
together.

Tolerances, from the arithmetic (u = 2^-24, half a step of fp32; h = eps / 2 of the 16-bit type, half
a step of the result):
  append  A rotated value x c - y s: table entries off by u each, one complex product of them (off
          by at most 4 u), two products and a sum (3 u of |x| + |y|): 7 u (|x| + |y|), taken as 10 u;
          then one rounding, h of the value (at least 2^-25, half fp16's smallest step).
  decode  A score s = scale sum_c q_c k_c accumulates its d products in fp32 in at most 16 steps,
          each off by at most 2 u of the running magnitude (the matrix unit may cut instead of
          rounding), and is scaled and shifted (2 u): |ds| <= e_s = 2^-19 (scale sum_c |q_c k_c|).
          A weight's relative error is e^{2 max e_s} - 1 (its own score and the reference's) plus
          2^-22 for the exponential and 2^-16 for the weight's two 16-bit parts; int8 adds one
          rounding of each value to fp16 (2^-11, or half of 2^-24).  Sums run in fp32 over at most n
          terms: n u / 16, as a lane adds every 16th tile.  Hence
          |do| <= (2 max e_s + 2^-15 + n u / 8) sum_t p_t |v_t| + h |o|, and
          |dlse| <= max e_s + 2^-20 + n u / 8 + 2 u |lse|.
"""
import numpy as np
import pytest
import torch

from oracle import kv_oracle as K
from rank_quantized_kv_decode_b200 import _lib as L
from rank_quantized_kv_decode_b200 import api

pytestmark = pytest.mark.gpu

ACT = {"bf16": torch.bfloat16, "f16": torch.float16, "int8": torch.bfloat16}
U = 2.0 ** -24
THETA = 10000.0


def half(fmt):
    return torch.finfo(ACT[fmt]).eps / 2


def f64(t):
    return t.detach().double().cpu().numpy()


class Case:
    """A cache of ragged sequences in shuffled pages, filled with NaN bytes before the appends."""

    def __init__(self, fmt, H, Hkv, d, lens, seed=0, spare=2, width=None, fill=0xFF):
        self.fmt, self.H, self.Hkv, self.d, self.lens = fmt, H, Hkv, d, list(lens)
        self.lay = api.kv_layout_init(api.make_kv_config(H, Hkv, d, fmt, THETA))
        self.olay = K.kv_page_layout(fmt, Hkv, d)
        B = len(lens)
        self.width = width or max(1, max(-(-n // 64) for n in lens))
        need = sum(-(-n // 64) for n in lens)
        self.kv = api.KvCache.create(self.lay, need + spare, B, self.width)
        self.kv.cache.fill_(fill)
        r = np.random.default_rng(seed)
        self.rng = r
        order = r.permutation(need + spare)
        table = np.zeros((B, self.width), np.int32)
        at = 0
        for b, n in enumerate(lens):
            m = -(-n // 64)
            table[b, :m] = order[at:at + m]
            at += m
        self.free = order[at:]
        self.table_np = table
        self.table = torch.from_numpy(table).cuda()
        self.len_t = torch.tensor(lens, dtype=torch.int32, device="cuda")

    def draw(self, n, heads, scale=1.0, shift=0.0):
        x = self.rng.standard_normal((n, heads, self.d)) * scale + shift
        return torch.from_numpy(x).to(ACT[self.fmt]).cuda()

    def fill(self, key_scale=1.0):
        """Appends every token of every sequence in one call; keys have a mean per channel."""
        n = sum(self.lens)
        if n == 0:
            return
        seq = np.concatenate([np.full(m, b) for b, m in enumerate(self.lens)]).astype(np.int32)
        pos = np.concatenate([np.arange(m) for m in self.lens]).astype(np.int32)
        self.k = self.draw(n, self.Hkv, key_scale, self.rng.standard_normal((1, self.Hkv, self.d)))
        self.v = self.draw(n, self.Hkv)
        self.append(self.k, self.v, seq, pos)

    def append(self, k, v, seq, pos, q=None, q_out=None):
        seq, pos = (torch.as_tensor(np.asarray(x, np.int32)).cuda() for x in (seq, pos))
        api.kv_append(self.lay, k, v, seq, pos, self.table, self.kv.cache, self.kv.rope, self.kv.status, q=q,
                      q_out=q_out)

    def pages(self):
        torch.cuda.synchronize()
        return self.kv.cache.cpu().numpy().reshape(-1, self.lay.page_bytes)

    def status(self):
        torch.cuda.synchronize()
        return self.kv.status.item()

    def decode(self, q, sel=None, lens=None, **kw):
        B = len(self.lens) if lens is None else lens.shape[0]
        out = torch.full((B, self.H, self.d), float("nan"), dtype=ACT[self.fmt], device="cuda")
        lse = torch.full((B, self.H), float("nan"), dtype=torch.float32, device="cuda")
        api.kv_decode(self.lay, q, self.kv.cache, self.table, self.len_t if lens is None else lens, out,
                      self.kv.decode_ws, self.kv.status, sel=sel, lse=lse, **kw)
        return out, lse

    def select(self, q, n_sel, first=0, last=1):
        sel = torch.full((len(self.lens), self.Hkv, n_sel), -7, dtype=torch.int32, device="cuda")
        api.kv_select(self.lay, q, self.kv.cache, self.table, self.len_t, sel, self.kv.status, keep_first=first,
                      keep_last=last)
        return sel

    def check(self, q, out, lse, sel=None, window=0, scale=None, skip=(), lens=None):
        """Every sequence against the oracle on the stored values (``skip``: pages of sequence 0 that
        are not read)."""
        cache, q, out, lse = self.pages(), f64(q), f64(out), f64(lse)
        G = self.H // self.Hkv
        sc = self.d ** -0.5 if scale is None else scale
        for b, n in enumerate(self.lens if lens is None else lens):
            for g in range(self.Hkv):
                pages = None
                if sel is not None:
                    pages = sel[b, g][sel[b, g] >= 0]
                elif skip and b == 0:
                    pages = np.array([i for i in range(-(-n // 64)) if i not in skip])
                k, v, pos = K.sequence(cache, self.olay, self.table_np[b], n, pages)
                ok = pos >= (max(0, n - window) if window else 0)
                k, v = k[g:g + 1, ok], v[g:g + 1, ok]
                qs = q[b, g * G:(g + 1) * G]
                want, wl, p, _ = K.attention(qs, k, v, sc)
                got, gl = out[b, g * G:(g + 1) * G], lse[b, g * G:(g + 1) * G]
                cnt = k.shape[1]
                if cnt == 0:
                    assert np.all(got == 0) and np.all(np.isneginf(gl))
                    continue
                es = 2.0 ** -19 * sc * np.max(np.einsum("hd,td->ht", np.abs(qs), np.abs(k[0])), 1)
                size = np.einsum("ht,td->hd", p, np.abs(v[0]))
                tol = (2 * es + 2.0 ** -15 + cnt * U / 8)[:, None] * size + half(self.fmt) * np.abs(want)
                tol += 2.0 ** -25 if self.fmt == "f16" else 2.0 ** -130
                if self.fmt == "int8":
                    tol += 2.0 ** -11 * size + 2.0 ** -25
                assert np.all(np.isfinite(got)), (b, g)
                bad = np.abs(got - want) / tol
                assert bad.max() <= 1, (b, g, n, float(bad.max()))
                dl = np.abs(gl - wl) / (es + 2.0 ** -20 + cnt * U / 8 + 2 * U * np.abs(wl))
                assert dl.max() <= 1, (b, g, n, float(dl.max()))


# ---------------------------------------------------------------------------------------- append
def rotated(x, pos):
    """fp64 rotation and the tolerance of its fp32 form."""
    x = f64(x)
    h = x.shape[-1] // 2
    pair = np.abs(x[..., :h]) + np.abs(x[..., h:])
    return K.rotate(x, pos, THETA), 10 * U * np.concatenate((pair, pair), -1)


def near16(got, want, tol, fmt):
    t = tol * (1 + half(fmt)) + half(fmt) * np.abs(want) + (2.0 ** -25 if fmt == "f16" else 0.0)
    bad = np.abs(got - want) - t
    assert np.all(np.isfinite(got)) and bad.max() <= 0, float(bad.max())


def near_codes(codes, scales, want, tol):
    """int8: the scale is the group's largest magnitude over 127 in fp16, each code the nearest."""
    g = np.abs(want).reshape(*want.shape[:-1], -1, 32)
    t = tol.reshape(g.shape)
    amax, dt = g.max(-1), t.max(-1)
    assert np.all(np.abs(scales - amax / 127) <= 2.0 ** -11 * amax / 127 + dt / 100 + 2.0 ** -25)
    got = codes * np.repeat(scales, 32, -1)
    # half a code step; a scale rounded down leaves the largest code at 127 up to 127 * 2^-11 steps short
    step = np.repeat(scales, 32, -1)
    assert np.all(np.abs(got - want) <= step * (0.5 + 2.0 ** -20) + tol + 2.0 ** -40)
    assert np.abs(codes).max() <= 127


@pytest.mark.parametrize("fmt", ["bf16", "f16", "int8"])
@pytest.mark.parametrize("H,Hkv,d,news", [
    (8, 2, 128, [1, 64, 65, 130]), (4, 4, 64, [63, 1, 3]), (10, 2, 128, [200]), (64, 1, 64, [5, 7]),
    (32, 32, 128, [2, 700]), (6, 1, 64, [2601, 2502])])  # the last: more tasks than warps
def test_append_stores_rotated_keys_values_and_bounds(fmt, H, Hkv, d, news):
    lens = [n + 61 * i for i, n in enumerate(news)]  # sequence i starts at position 61 i
    c = Case(fmt, H, Hkv, d, lens, seed=3)
    before = c.pages().copy()
    seq = np.concatenate([np.full(n, b) for b, n in enumerate(news)])
    pos = np.concatenate([np.arange(m - n, m) for n, m in zip(news, lens)])
    order = c.rng.permutation(len(seq))  # tokens in any order
    seq, pos = seq[order], pos[order]
    n = len(seq)
    # a fused projection: q, k and v side by side
    qkv = c.draw(n, H + 2 * Hkv)
    q, k, v = qkv[:, :H], qkv[:, H:H + Hkv], qkv[:, H + Hkv:]
    q_out = torch.empty(n, H, d, dtype=ACT[fmt], device="cuda")
    c.append(k, v, seq, pos, q=q, q_out=q_out)
    assert c.status() == 0
    near16(f64(q_out), *rotated(q, pos), fmt)
    cache = c.pages()
    page, slot = c.table_np[seq, pos // 64], pos % 64
    want, tol = rotated(k, pos)
    if fmt == "int8":
        kc, vc, ks, vs = K.read_raw(cache, c.olay)
        near_codes(kc[page, :, slot], ks[page, :, slot], want, tol)
        wc, ws = K.quantise(f64(v))
        assert np.array_equal(vc[page, :, slot], wc) and np.array_equal(vs[page, :, slot], ws)
    else:
        keys, values = K.read_tokens(cache, c.olay)
        near16(keys[page, :, slot], want, tol, fmt)
        assert np.array_equal(values[page, :, slot], f64(v))
    # bounds of the pages whose slot 63 was written are exact for their stored keys; the keys that no
    # call stored are NaN bytes, which no bound takes
    done = c.table_np[seq, pos // 64][slot == 63]
    keys, _ = K.read_tokens(cache, c.olay)
    bounds = K.read_bounds(cache, c.olay)
    for p in done:
        lo, hi = np.nanmin(keys[p], 1), np.nanmax(keys[p], 1)
        if fmt == "int8":  # fill bytes 0xFF are code -1 under a NaN scale: NaN as well
            lo, hi = (f64(torch.from_numpy(x).bfloat16()) for x in (lo, hi))
        assert np.array_equal(bounds[p, :, 0], lo) and np.array_equal(bounds[p, :, 1], hi)
    # nothing else changed: blank what was written, on both sides
    for img in (before, cache):
        img[done, :c.olay["off_heads"]] = 0
        t = img[:, c.olay["off_heads"]:].reshape(-1, Hkv, c.olay["head_bytes"])
        row = d if fmt == "int8" else 2 * d
        offs = [(0, row), (c.olay["off_v"], row)]
        if fmt == "int8":
            offs += [(c.olay["off_ks"], d // 16), (c.olay["off_vs"], d // 16)]
        for p, s in zip(page, slot):
            for o, w in offs:
                t[p, :, o + s * w:o + (s + 1) * w] = 0
        img[:, c.olay["off_heads"]:] = t.reshape(img.shape[0], -1)
    assert np.array_equal(before, cache)


@pytest.mark.parametrize("fmt", ["bf16", "f16", "int8"])
def test_token_by_token_and_read_back_equal_one_call(fmt):
    a, b = (Case(fmt, 4, 2, 64, [130, 67], seed=5) for _ in range(2))
    a.fill()
    n0 = 130
    for i in range(130):  # a step for both sequences while the second lasts
        rows = [i] + ([n0 + i] if i < 67 else [])
        b.append(a.k[rows], a.v[rows], [0, 1][:len(rows)], [i] * len(rows))
    assert np.array_equal(a.pages(), b.pages()) and a.status() == 0 and b.status() == 0
    seq = torch.tensor([0] * 130 + [1] * 67, dtype=torch.int32, device="cuda")
    pos = torch.cat([torch.arange(130), torch.arange(67)]).int().cuda()
    ko, vo = (torch.full((197, 2, 64), 7.0, dtype=ACT[fmt], device="cuda") for _ in range(2))
    api.kv_gather(a.lay, a.kv.cache, seq, pos, a.table, ko, vo, a.kv.status)
    keys, values = K.read_tokens(a.pages(), a.olay)
    page, slot = a.table_np[seq.cpu(), pos.cpu() // 64], pos.cpu().numpy() % 64
    for got, all_ in ((ko, keys), (vo, values)):
        want = torch.from_numpy(all_[page, :, slot]).float().to(ACT[fmt])
        assert torch.equal(got.cpu(), want)


@pytest.mark.parametrize("fmt", ["bf16", "f16", "int8"])
def test_one_launch_and_two_leave_the_same_pages(fmt):
    # 32 tokens are stored and bounded in one launch, 33 in two; and in calls of 100
    cs = [Case(fmt, 4, 2, 128, [400], seed=5) for _ in range(3)]
    k, v = cs[0].draw(400, 2), cs[0].draw(400, 2)
    for c, cut in zip(cs, ([0, 400], list(range(0, 385, 32)) + [400], [0, 100, 200, 300, 400])):
        for a, b in zip(cut, cut[1:]):
            c.append(k[a:b], v[a:b], np.zeros(b - a), np.arange(a, b))
    assert np.array_equal(cs[0].pages(), cs[1].pages()) and np.array_equal(cs[0].pages(), cs[2].pages())


def test_int8_codes_at_the_edges():
    """Values stored as they are: quotients at and next to a half, groups of zeros, of subnormals, of one
    large value, beyond fp16's largest scale, and an infinity; codes and scales are those of the oracle."""
    c = Case("int8", 1, 1, 64, [300], seed=3)
    r = c.rng
    x = r.standard_normal((300, 64)).astype(np.float32)
    # scale 1: the largest is 127, the others whole numbers and halves (ties to even)
    x[:100] = r.integers(-254, 255, (100, 64)) / 2
    x[:100, ::32] = 127
    # other scales: the largest sets it, the others are halves of it before their rounding to bf16
    for i in range(100, 200):
        s = np.float32(np.float16(2.0 ** r.uniform(-20, 8)))
        x[i] = (r.integers(-126, 127, 64) + 0.5) * s
        x[i, ::32] = 127 * s
    x[200] = 0
    x[201, :32], x[201, 32:] = 0, 1e-8
    x[202] = 1e-38
    x[203], x[203, 5] = 1e-3, 3e4
    x[204], x[204, 7] = 1e6, -3e38
    x[205, 9] = np.inf
    v = torch.from_numpy(x)[:, None].bfloat16().cuda()
    c.append(v, v, np.zeros(300), np.arange(300))
    _, codes, _, scales = K.read_raw(c.pages(), c.olay)
    with np.errstate(over="ignore"):
        wc, ws = K.quantise(f64(v))
    page, slot = c.table_np[0][np.arange(300) // 64], np.arange(300) % 64
    assert np.array_equal(scales[page, :, slot], ws)
    assert np.array_equal(codes[page, :, slot], wc)


@pytest.mark.parametrize("fmt", ["bf16", "f16", "int8"])
@pytest.mark.parametrize("batch", [5, 32, 33, 300])
def test_a_batch_that_completes_its_pages_together(fmt, batch):
    # one launch up to 32 tokens, two beyond; every token stands in slot 63
    c = Case(fmt, 4, 2, 64, [64] * batch, seed=batch)
    n = 64 * batch
    k, v = c.draw(n, 2), c.draw(n, 2)
    seq, pos = np.repeat(np.arange(batch), 64), np.tile(np.arange(64), batch)
    early, last = np.flatnonzero(pos < 63), np.flatnonzero(pos == 63)
    c.append(k[early], v[early], seq[early], pos[early])
    assert np.all(c.pages()[:, :c.olay["off_heads"]] == 0xFF)  # no page is complete, no bounds are written
    c.append(k[last], v[last], seq[last], pos[last])
    keys, _ = K.read_tokens(c.pages(), c.olay)
    b = K.read_bounds(c.pages(), c.olay)
    p = c.table_np[:, 0]
    lo, hi = keys[p].min(2), keys[p].max(2)
    if fmt == "int8":
        lo, hi = (f64(torch.from_numpy(x).bfloat16()) for x in (lo, hi))
    assert np.array_equal(b[p][:, :, 0], lo) and np.array_equal(b[p][:, :, 1], hi)


def test_rewriting_slot_63_renews_the_bounds():
    c = Case("bf16", 2, 1, 64, [64])
    c.fill()
    c.append(c.k[:1] * 100, c.v[:1], [0], [7])
    c.append(c.k[63:], c.v[63:], [0], [63])
    keys, _ = K.read_tokens(c.pages(), c.olay)
    b = K.read_bounds(c.pages(), c.olay)[c.table_np[0, 0]]
    assert np.array_equal(b[:, 0], keys[c.table_np[0, 0]].min(1)) and np.array_equal(b[:, 1], keys[c.table_np[0, 0]].max(1))


def test_far_positions_and_queries_in_place():
    far = 1 << 20
    c = Case("f16", 4, 1, 64, [1], width=far // 64)
    pos = np.array([far - 1, far - 64, far // 2 + 1, 127, 128])
    c.table[0, :] = torch.arange(far // 64, dtype=torch.int32).cuda() % 3
    c.table_np = c.table.cpu().numpy()
    pos = pos[np.unique(c.table_np[0, pos // 64] * 64 + pos % 64, return_index=True)[1]]
    q, k, v = c.draw(len(pos), 4), c.draw(len(pos), 1), c.draw(len(pos), 1)
    want, tol = rotated(q, pos)
    c.append(k, v, np.zeros(len(pos)), pos, q=q, q_out=q)
    near16(f64(q), want, tol, "f16")
    keys, _ = K.read_tokens(c.pages(), c.olay)
    near16(keys[c.table_np[0, pos // 64], :, pos % 64], *rotated(k, pos), "f16")


def test_append_and_gather_flag_and_skip_bad_tokens():
    c = Case("bf16", 2, 1, 64, [64, 64], width=2)
    c.table[0, 1] = c.kv.num_pages  # a page outside the pool
    c.table[1, 1] = -1
    before = c.pages().copy()
    seq = np.array([0, 2, -1, 0, 0, 0, 1])
    pos = np.array([-1, 0, 0, 128, 64, 127, 127])
    q, k = c.draw(7, 2), c.draw(7, 1)
    q_out = torch.full_like(q, 7.0)
    c.append(k, k, seq, pos, q=q, q_out=q_out)
    assert c.status() == L.DEV_BOUNDS
    assert np.array_equal(before, c.pages())
    inside = (pos >= 0) & (pos < 128)
    want, tol = rotated(q, np.where(inside, pos, 0))
    near16(f64(q_out)[inside], want[inside], tol[inside], "bf16")
    assert np.all(f64(q_out)[~inside] == 0)
    c.kv.status.zero_()
    ko, vo = (torch.full((7, 1, 64), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    api.kv_gather(c.lay, c.kv.cache, torch.from_numpy(seq).int().cuda(), torch.from_numpy(pos).int().cuda(), c.table,
                  ko, vo, c.kv.status)
    assert c.status() == L.DEV_BOUNDS and not ko.any() and not vo.any()


# ---------------------------------------------------------------------------------------- decode
LENS = [0, 1, 15, 16, 17, 63, 64, 65, 128, 1000, 0, 449]


@pytest.mark.parametrize("fmt", ["bf16", "f16", "int8"])
@pytest.mark.parametrize("H,Hkv,d", [(8, 2, 128), (4, 4, 64), (10, 2, 128), (3, 1, 64), (32, 4, 64), (32, 2, 128),
                                     (20, 2, 64), (64, 1, 128)])
def test_decode_matches_oracle(fmt, H, Hkv, d):
    c = Case(fmt, H, Hkv, d, LENS, seed=H + d)
    c.fill()
    q = c.draw(len(LENS), H, 1.5)
    out, lse = c.decode(q)
    assert c.status() == 0
    c.check(q, out, lse)
    again, lse2 = c.decode(q)
    assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("ctas", [1, 2, 5, 37, 296])
@pytest.mark.parametrize("fmt", ["bf16", "int8"])
def test_decode_at_any_split(fmt, ctas):
    c = Case(fmt, 6, 2, 128, [300, 0, 1, 700, 64], seed=2)
    c.fill()
    q = c.draw(5, 6, 1.5)
    out, lse = c.decode(q, max_ctas=ctas)
    assert c.status() == 0
    c.check(q, out, lse)


@pytest.mark.parametrize("batch", [1, 31, 32, 33, 70])
def test_decode_batches_around_a_warp(batch):
    lens = [(37 * i) % 150 for i in range(batch)]
    lens[-1] = 91
    c = Case("bf16", 2, 2, 64, lens, seed=batch)
    c.fill()
    q = c.draw(batch, 2, 1.5)
    out, lse = c.decode(q)
    c.check(q, out, lse)


@pytest.mark.parametrize("fmt,d", [("bf16", 128), ("f16", 64), ("int8", 128), ("int8", 64)])
@pytest.mark.parametrize("window", [1, 16, 63, 64, 65, 200, 100000])
def test_window(fmt, d, window):
    c = Case(fmt, 8, 2, d, [1, 64, 65, 1000, 0, 130], seed=9)
    c.fill()
    # what lies before the window may have been given away: NaN there
    img = c.pages().copy()
    for b, n in enumerate(c.lens):
        for i in range(max(0, n - window) // 64):
            img[c.table_np[b, i]] = 0xFF
    c.kv.cache.copy_(torch.from_numpy(img.reshape(-1)))
    q = c.draw(6, 8, 1.5)
    out, lse = c.decode(q, window=window)
    assert c.status() == 0
    c.check(q, out, lse, window=window)


@pytest.mark.parametrize("fmt", ["bf16", "f16", "int8"])
@pytest.mark.parametrize("scale", [0.02, 0.5, 4.0])
def test_sharp_and_flat_softmax(fmt, scale):
    c = Case(fmt, 8, 2, 64, [1500, 77], seed=4)
    c.fill(key_scale=2.0)
    q = c.draw(2, 8, 3.0)
    out, lse = c.decode(q, scale=scale)
    c.check(q, out, lse, scale=float(np.float32(scale)))


def test_rising_scores_and_a_long_flat_tail():
    # the reference moves at almost every tile; and 60000 tokens of weight 2^-18 against one of weight 1
    for case in range(2):
        n = 2000 if case == 0 else 60000
        c = Case("f16", 1, 1, 64, [n], seed=6)
        x = np.zeros((n, 1, 64))
        x[:, 0, 63] = np.arange(n) / 8.0 if case == 0 else 0.0  # channel 63 turns slowest
        if case == 1:
            x[n - 1, 0, 63] = 18.0
        k = torch.from_numpy(x).half().cuda()
        v = torch.ones(n, 1, 64, dtype=torch.float16, device="cuda")
        v[n - 1] = -1.0
        c.append(k, v, np.zeros(n), np.arange(n))
        keys, _, _ = K.sequence(c.pages(), c.olay, c.table_np[0], n)
        q = torch.zeros(1, 1, 64, dtype=torch.float16, device="cuda")
        # along the stored direction of the last key
        q[0, 0] = torch.from_numpy(keys[0, -1] / np.linalg.norm(keys[0, -1])).half().cuda()
        out, lse = c.decode(q, scale=float(np.float32(np.log(2.0))))
        c.check(q, out, lse, scale=float(np.float32(np.log(2.0))))


def test_queries_of_any_magnitude():
    c = Case("int8", 4, 1, 64, [200], seed=8)
    c.fill()
    base = c.draw(1, 4)
    for e in (-60, -20, 0, 12):
        q = base * 2.0 ** e
        q[0, 3] = 0
        s = float(2.0 ** -e)
        out, lse = c.decode(q, scale=s)
        c.check(q, out, lse, scale=s)


def test_bad_pages_and_lengths_are_flagged_and_skipped():
    c = Case("bf16", 8, 2, 128, [400, 100], seed=1)
    c.fill()
    q = c.draw(2, 8, 1.5)
    keep = c.table.clone()
    c.table[0, 2], c.table[0, 5] = -3, c.kv.num_pages
    out, lse = c.decode(q)
    assert c.status() == L.DEV_BOUNDS
    c.check(q, out, lse, skip=(2, 5))
    c.table[0, :] = -1  # nothing left of sequence 0
    c.kv.status.zero_()
    out, lse = c.decode(q)
    assert c.status() == L.DEV_BOUNDS
    assert not out[0].any() and torch.isneginf(lse[0]).all()
    c.table.copy_(keep)
    c.kv.status.zero_()
    # a length beyond the block table is cut to it, a negative one is empty
    lens = torch.tensor([c.width * 64 + 9, -5], dtype=torch.int32, device="cuda")
    c.lens = [c.width * 64, 0]
    img = c.pages().copy()
    img[c.table_np[0, -1]] = img[c.table_np[0, 0]]
    c.kv.cache.copy_(torch.from_numpy(img.reshape(-1)))
    out, lse = c.decode(q, lens=lens)
    assert c.status() == L.DEV_BOUNDS
    c.check(q, out, lse)
    c.kv.status.zero_()
    c.decode(q, lens=torch.tensor([-1, -5], dtype=torch.int32, device="cuda"))
    assert c.status() == L.DEV_BOUNDS


def test_infinite_and_nan_values_reach_only_their_rows():
    c = Case("bf16", 2, 2, 64, [100, 100], seed=1)
    c.fill()
    q = c.draw(2, 2)
    want, _ = c.decode(q)
    k = c.k[50:51].clone()
    v = c.v[50:51].clone()
    v[0, 0, 5] = float("nan")
    v[0, 1, 7] = float("inf")
    c.append(k, v, [0], [50])
    out, _ = c.decode(q)
    assert torch.equal(out[1], want[1])
    assert not torch.isfinite(out[0, 0, 5]) and not torch.isfinite(out[0, 1, 7])
    ok = torch.ones_like(out[0], dtype=torch.bool)
    ok[0, 5] = ok[1, 7] = False
    assert torch.equal(out[0][ok], want[0][ok])


@pytest.mark.parametrize("fmt", ["bf16", "int8"])
def test_workspace_needs_no_initial_values(fmt):
    """Whatever the workspace holds, a count of another call's or nothing sensible, results are the same
    bits; and a call of other sizes between changes nothing."""
    c = Case(fmt, 8, 2, 128, [3000, 17, 20000, 640], seed=13)
    c.fill()
    o = Case("f16", 4, 4, 64, [5000, 100], seed=14)
    o.fill()
    q, qo = c.draw(4, 8, 1.5), o.draw(2, 4)
    out, lse = c.decode(q)
    c.check(q, out, lse)
    ws = c.kv.decode_ws
    for i, fill in enumerate((0x00, 0xFF, 0x80, None)):
        if fill is None:
            ws.copy_(torch.randint(0, 256, ws.shape, dtype=torch.uint8, device="cuda"))
        else:
            ws.fill_(fill)
        for _ in range(3):
            again, lse2 = c.decode(q)
            assert torch.equal(out, again) and torch.equal(lse, lse2), (i, _)
            o.kv.decode_ws = ws
            o.decode(qo)


# ---------------------------------------------------------------------------------------- selection
@pytest.mark.parametrize("fmt", ["bf16", "f16", "int8"])
@pytest.mark.parametrize("H,Hkv,d", [(8, 2, 128), (4, 4, 64), (10, 2, 128), (3, 1, 64), (32, 2, 64), (20, 1, 128),
                                     (4, 2, 64)])
def test_select_matches_oracle(fmt, H, Hkv, d):
    lens = [0, 1, 64, 65, 449, 64 * 40, 64 * 97 - 5, 64 * 33 + 1]
    c = Case(fmt, H, Hkv, d, lens, seed=H * d)
    c.fill()
    q = c.draw(len(lens), H, 1.5)
    bounds = K.read_bounds(c.pages(), c.olay)
    for n_sel, first, last in ((1, 0, 1), (3, 1, 2), (7, 1, 1), (40, 2, 3), (200, 0, 1)):
        sel = c.select(q, n_sel, first, last).cpu().numpy()
        assert c.status() == 0
        for b, n in enumerate(lens):
            s = K.page_scores(f64(q)[b], bounds[c.table_np[b, :-(-n // 64)]])
            for g in range(Hkv):
                assert np.array_equal(sel[b, g], K.choose(s[g], n, n_sel, first, last)), (n_sel, b, g)


@pytest.mark.parametrize("pages", [5, 256, 257, 600])
def test_equal_pages_are_chosen_from_the_lowest(pages):
    c = Case("bf16", 2, 1, 64, [64 * pages], seed=2)
    k = c.draw(64, 1)
    c.append(k, k, np.zeros(64), np.arange(64))
    img = c.pages().copy()
    img[:] = img[c.table_np[0, 0]]
    better = c.table_np[0, pages // 2]  # one page above the others
    hi = img[better].copy()
    bits = torch.from_numpy(hi[:c.olay["off_heads"]].view(np.int16).copy()).view(torch.bfloat16)
    bits = torch.cat((bits[:64] - 1, bits[64:] + 1))
    hi[:c.olay["off_heads"]] = bits.view(torch.int16).numpy().view(np.uint8)
    img[better] = hi
    c.kv.cache.copy_(torch.from_numpy(img.reshape(-1)))
    q = c.draw(1, 2)
    n_sel = pages - 1
    sel = c.select(q, n_sel, 0, 1).cpu().numpy()[0, 0]
    want = sorted(set(range(pages - 2)) | {pages // 2, pages - 1})
    assert list(sel) == want


@pytest.mark.parametrize("what", [float("nan"), float("inf"), -float("inf")])
def test_select_with_numbers_that_are_none_still_gives_pages(what):
    c = Case("bf16", 4, 2, 64, [64 * 40], seed=2)
    c.fill()
    k = c.k[:5].clone()
    k[:, :, 3] = what
    for i in range(5):  # pages 0, 7, ... with slot 63 again
        p = 64 * 7 * i
        c.append(torch.cat((k[i:i + 1], c.k[p + 63:p + 64])), torch.cat((c.v[:1], c.v[:1])), [0, 0], [p + 5, p + 63])
    for q in (c.draw(1, 4), torch.full((1, 4, 64), what, dtype=torch.bfloat16, device="cuda")):
        for n_sel in (2, 9, 39):
            sel = c.select(q, n_sel, 1, 1).cpu().numpy()[0]
            for g in range(2):
                assert np.all(np.diff(sel[g]) > 0) and sel[g, 0] == 0 and sel[g, -1] == 39
    assert c.status() == 0


@pytest.mark.parametrize("n_sel,first,last", [(50, 1, 2), (1000, 0, 1), (16383, 2, 3)])
def test_select_over_the_longest_table_with_many_equal_pages(n_sel, first, last):
    """A million tokens: 16384 places that share 90 pages, so that every score stands many times and the
    border falls among equal ones; then attention over the choice."""
    pages = 16384
    c = Case("bf16", 4, 1, 64, [64 * 90], seed=21)
    c.fill()
    order = np.concatenate([c.table_np[0], c.table_np[0][c.rng.integers(0, 90, pages - 90)]])
    c.table_np = order[None].astype(np.int32)
    c.table = torch.from_numpy(c.table_np).cuda()
    c.lens = [pages * 64 - 13]
    c.len_t = torch.tensor(c.lens, dtype=torch.int32, device="cuda")
    q = c.draw(1, 4, 1.5)
    sel = c.select(q, n_sel, first, last).cpu().numpy()
    s = K.page_scores(f64(q)[0], K.read_bounds(c.pages(), c.olay)[c.table_np[0]])
    assert np.array_equal(sel[0, 0], K.choose(s[0], c.lens[0], n_sel, first, last))
    assert c.status() == 0
    out, lse = c.decode(q, sel=torch.from_numpy(sel).int().cuda())
    c.check(q, out, lse, sel=sel)


def test_select_flags_a_bad_page_and_ranks_it_last():
    c = Case("bf16", 4, 2, 64, [64 * 9], seed=2)
    c.fill()
    q = c.draw(1, 4)
    bounds = K.read_bounds(c.pages(), c.olay)
    s = K.page_scores(f64(q)[0], bounds[c.table_np[0]])
    s[:, [1, 4]] = -np.inf
    c.table[0, 1], c.table[0, 4] = -1, 1 << 30
    sel = c.select(q, 7, 0, 1).cpu().numpy()
    assert c.status() == L.DEV_BOUNDS
    for g in range(2):
        assert np.array_equal(sel[0, g], K.choose(s[g], 64 * 9, 7, 0, 1))


@pytest.mark.parametrize("fmt,d,H,Hkv", [("bf16", 128, 8, 2), ("f16", 64, 10, 2), ("int8", 128, 32, 2), ("int8", 64, 4, 4)])
def test_attention_over_a_selection(fmt, d, H, Hkv):
    lens = [0, 30, 64 * 5, 1000, 2111]
    c = Case(fmt, H, Hkv, d, lens, seed=7)
    c.fill()
    q = c.draw(5, H, 1.5)
    sel = np.full((5, Hkv, 6), -1, np.int32)
    for b, n in enumerate(lens):
        P = -(-n // 64)
        for g in range(Hkv):
            m = min(P, 6) - (g if P > 6 else 0)  # fewer than the places, for some heads
            sel[b, g, :m] = np.sort(c.rng.choice(P, m, replace=False)) if m else []
    c.rng.shuffle(sel[3, 0])  # any order, -1 anywhere
    out, lse = c.decode(q, sel=torch.from_numpy(sel).cuda())
    assert c.status() == 0
    c.check(q, out, lse, sel=sel)
    # places outside the sequence are flagged and skipped; all of them -1: nothing
    bad = sel.copy()
    bad[4, 0, 0], bad[4, 0, 1] = 33 + 1, -2
    out, lse = c.decode(q, sel=torch.from_numpy(bad).cuda())
    assert c.status() == L.DEV_BOUNDS
    bad[4, 0, :2] = -1
    c.check(q, out, lse, sel=bad)
    none = torch.full((5, Hkv, 6), -1, dtype=torch.int32, device="cuda")
    out, lse = c.decode(q, sel=none)
    assert not out.any() and torch.isneginf(lse).all()


# ---------------------------------------------------------------------------------------- together
@pytest.mark.parametrize("fmt", ["bf16", "f16", "int8"])
def test_decode_steps_append_select_attend(fmt):
    """A generation loop: every step appends one token per sequence (from a fused projection), attends
    to everything, chooses pages and attends to those."""
    start, steps = [60, 1, 700], 70
    c = Case(fmt, 8, 2, 64, [n + steps for n in start], seed=11)
    full = list(c.lens)
    c.lens = list(start)
    c.fill()
    for i in range(steps):
        lens = [n + i + 1 for n in start]
        qkv = c.draw(3, 12)
        q = torch.empty(3, 8, 64, dtype=ACT[fmt], device="cuda")
        c.append(qkv[:, 8:10], qkv[:, 10:], [0, 1, 2], [n - 1 for n in lens], q=qkv[:, :8], q_out=q)
        c.lens, c.len_t = lens, torch.tensor(lens, dtype=torch.int32, device="cuda")
        if i % 9 and i != 3:  # 700 + 4 tokens complete a page, 60 + 4 too
            continue
        out, lse = c.decode(q)
        c.check(q, out, lse)
        sel = c.select(q, 5, 1, 1)
        out, lse = c.decode(q, sel=sel)
        bounds = K.read_bounds(c.pages(), c.olay)
        s = sel.cpu().numpy()
        for b, n in enumerate(lens):
            sc = K.page_scores(f64(q)[b], bounds[c.table_np[b, :-(-n // 64)]])
            for g in range(2):
                assert np.array_equal(s[b, g], K.choose(sc[g], n, 5, 1, 1))
        c.check(q, out, lse, sel=s)
    assert c.status() == 0 and full == lens


def test_a_captured_step_replays_at_other_lengths():
    c = Case("bf16", 8, 2, 128, [500, 900, 64], seed=3)
    c.fill()
    full = list(c.lens)
    qkv = c.draw(3, 12)
    q = torch.empty(3, 8, 128, dtype=torch.bfloat16, device="cuda")
    out, sp = torch.empty_like(q), torch.empty_like(q)
    lse = torch.empty(3, 8, device="cuda")
    sel = torch.empty(3, 2, 4, dtype=torch.int32, device="cuda")
    seq = torch.arange(3, dtype=torch.int32, device="cuda")
    pos = torch.zeros(3, dtype=torch.int32, device="cuda")

    def step():
        api.kv_append(c.lay, qkv[:, 8:10], qkv[:, 10:], seq, pos, c.table, c.kv.cache, c.kv.rope, c.kv.status,
                      q=qkv[:, :8], q_out=q)
        api.kv_decode(c.lay, q, c.kv.cache, c.table, c.len_t, out, c.kv.decode_ws, c.kv.status, lse=lse)
        api.kv_select(c.lay, q, c.kv.cache, c.table, c.len_t, sel, c.kv.status)
        api.kv_decode(c.lay, q, c.kv.cache, c.table, c.len_t, sp, c.kv.decode_ws, c.kv.status, sel=sel)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    c.len_t.copy_(torch.tensor(full))
    pos.copy_(c.len_t - 1)
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for lens in ([500, 900, 64], [128, 1, 0], [65, 700, 63]):
        c.lens = lens
        c.len_t.copy_(torch.tensor(lens))
        pos.copy_((c.len_t - 1).clamp(min=0))
        qkv.copy_(c.draw(3, 12))
        graph.replay()
        c.check(q, out, lse)
        eager = torch.empty_like(out)
        api.kv_decode(c.lay, q, c.kv.cache, c.table, c.len_t, eager, c.kv.decode_ws, c.kv.status)
        assert torch.equal(eager, out)
        s2 = torch.empty_like(sel)
        api.kv_select(c.lay, q, c.kv.cache, c.table, c.len_t, s2, c.kv.status)
        assert torch.equal(s2, sel)
    assert c.status() == 0


def test_two_streams_with_a_workspace_each():
    cs = [Case("bf16", 32, 8, 128, [3000 - 700 * i, 5000], seed=i) for i in range(2)]
    for c in cs:
        c.fill()
    qs = [c.draw(2, 32, 1.5) for c in cs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cs]
    outs = [(torch.empty_like(q), torch.empty(2, 32, device="cuda")) for q in qs]
    torch.cuda.synchronize()
    for _ in range(20):
        for c, q, (o, l), st in zip(cs, qs, outs, streams):
            api.kv_decode(c.lay, q, c.kv.cache, c.table, c.len_t, o, c.kv.decode_ws, c.kv.status, lse=l, stream=st)
    torch.cuda.synchronize()
    for c, q, (o, l) in zip(cs, qs, outs):
        c.check(q, o, l)


def test_pages_beyond_four_gigabytes():
    # 20000 pages of 266 kB: the sequence's pages lie on both sides of 2^32 bytes and at the end
    H, Hkv, d = 8, 8, 128
    lay = api.kv_layout_init(api.make_kv_config(H, Hkv, d, "bf16", THETA))
    n = 20000
    c = Case("bf16", H, Hkv, d, [200], seed=5)
    kv = api.KvCache.create(lay, n, 1, c.width)
    assert kv.cache.numel() > 1 << 32
    far = np.array([n - 1, 0, (1 << 32) // lay.page_bytes, n // 2], np.int32)
    c.kv = kv
    c.table_np = far[None]
    c.table = torch.from_numpy(c.table_np).cuda()
    c.fill()
    q = c.draw(1, H, 1.5)
    out, lse = c.decode(q)
    sel = c.select(q, 2)
    out2, lse2 = c.decode(q, sel=sel)
    assert c.status() == 0
    rows = kv.cache.view(n, -1)[torch.from_numpy(far).long().cuda()]
    kv.cache = rows.reshape(-1).clone()
    c.table_np = np.arange(4, dtype=np.int32)[None]
    c.check(q, out, lse)
    s = K.page_scores(f64(q)[0], K.read_bounds(c.pages(), c.olay))
    got = sel.cpu().numpy()
    for g in range(Hkv):
        assert np.array_equal(got[0, g], K.choose(s[g], 200, 2, 0, 1))
    c.check(q, out2, lse2, sel=got)


def test_strided_rows_and_single_tokens():
    # rows of a wider tensor, and one token whose stride says nothing
    c = Case("bf16", 4, 2, 64, [3], seed=5)
    wide = c.draw(3, 40)
    c.append(wide[:, 3:5], wide[:, 30:32], [0, 0, 0], [0, 1, 2])
    d2 = Case("bf16", 4, 2, 64, [3], seed=5)
    for i in range(3):
        d2.append(wide[i:i + 1, 3:5], wide[i:i + 1, 30:32], [0], [i])
    assert np.array_equal(c.pages(), d2.pages())
    _, values = K.read_tokens(c.pages(), c.olay)
    assert np.array_equal(values[c.table_np[0, 0], :, :3].transpose(1, 0, 2), f64(wide[:, 30:32]))


def test_binding_refuses_rows_the_library_cannot_take():
    c = Case("bf16", 4, 2, 64, [3])
    x = torch.zeros(3 * 2 * 68 + 1, dtype=torch.bfloat16, device="cuda")
    odd = x[1:1 + 3 * 128].view(3, 2, 64)  # 2-byte aligned
    good = torch.zeros(3, 2, 64, dtype=torch.bfloat16, device="cuda")
    for k, v in ((odd, good), (good, odd)):
        with pytest.raises(L.StarkvError) as e:
            c.append(k, v, [0, 0, 0], [0, 1, 2])
        assert e.value.status == L.ERR_INVALID_ARG
    ragged = x[:3 * 2 * 68].view(3, 136)[:, :128].as_strided((3, 2, 64), (132, 64, 1))
    with pytest.raises(L.StarkvError):
        c.append(ragged, good, [0, 0, 0], [0, 1, 2])
    assert c.status() == 0
