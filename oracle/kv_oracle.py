"""fp64 reference of the plain key-value cache: page layout, append (rotation, storage, bounds),
choice of pages, attention of one token.

TEST INFRASTRUCTURE, like the rest of this package.  Caches are uint8 arrays [pages][page_bytes].
"""
from __future__ import annotations

import numpy as np

from . import starkv_oracle as O

PAGE = 64
GROUP = 32


def kv_page_layout(fmt: str, n_kv_heads: int, d: int) -> dict:
    """Offsets of a page: bounds [n_kv_heads][2][d] of 16 bits, then per KV head the keys [64][d], the
    values [64][d] and, for int8, their fp16 scales [64][d/32]."""
    el = 1 if fmt == "int8" else 2
    scales = PAGE * (d // GROUP) * 2 if fmt == "int8" else 0
    keys = PAGE * d * el
    off_heads = n_kv_heads * 2 * d * 2
    head = 2 * keys + 2 * scales
    return dict(fmt=fmt, n_kv_heads=n_kv_heads, d=d, off_heads=off_heads, head_bytes=head, off_v=keys,
                off_ks=2 * keys if scales else -1, off_vs=2 * keys + scales if scales else -1,
                page_bytes=off_heads + n_kv_heads * head, token_bytes=n_kv_heads * head // PAGE)


def from_bits(bits, fmt: str) -> np.ndarray:
    """fp64 values of 16-bit patterns (bf16, or fp16 for fmt "f16")."""
    bits = np.ascontiguousarray(bits, dtype=np.uint16)
    if fmt == "f16":
        return bits.view(np.float16).astype(np.float64)
    return (bits.astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def read_bounds(cache, lay: dict) -> np.ndarray:
    """Bounds of every page, fp64 [pages][n_kv_heads][2][d]."""
    n = cache.shape[0]
    raw = np.ascontiguousarray(cache[:, :lay["off_heads"]]).view(np.uint16)
    return from_bits(raw, lay["fmt"]).reshape(n, lay["n_kv_heads"], 2, lay["d"])


def read_raw(cache, lay: dict):
    """int8: (key codes, value codes [pages][heads][64][d] int64, key scales, value scales fp64)."""
    n, H, d = cache.shape[0], lay["n_kv_heads"], lay["d"]
    t = cache[:, lay["off_heads"]:].reshape(n, H, lay["head_bytes"])
    size = PAGE * d

    def codes(o):
        return np.ascontiguousarray(t[:, :, o:o + size]).view(np.int8).reshape(n, H, PAGE, d).astype(np.int64)

    def scales(o):
        b = PAGE * (d // GROUP) * 2
        return np.ascontiguousarray(t[:, :, o:o + b]).view(np.float16).reshape(n, H, PAGE, d // GROUP).astype(np.float64)

    return codes(0), codes(lay["off_v"]), scales(lay["off_ks"]), scales(lay["off_vs"])


def read_tokens(cache, lay: dict):
    """Stored keys and values, fp64 [pages][n_kv_heads][64][d]."""
    n, H, d = cache.shape[0], lay["n_kv_heads"], lay["d"]
    if lay["fmt"] == "int8":
        kc, vc, ks, vs = read_raw(cache, lay)
        return kc * np.repeat(ks, GROUP, 3), vc * np.repeat(vs, GROUP, 3)
    t = cache[:, lay["off_heads"]:].reshape(n, H, lay["head_bytes"])
    out = []
    for o in (0, lay["off_v"]):
        raw = np.ascontiguousarray(t[:, :, o:o + 2 * PAGE * d]).view(np.uint16)
        out.append(from_bits(raw, lay["fmt"]).reshape(n, H, PAGE, d))
    return out[0], out[1]


def sequence(cache, lay: dict, table_row, length: int, pages=None):
    """Keys, values [n_kv_heads][tokens][d] of a sequence and their positions; ``pages`` (page indices
    of the sequence) restricts them."""
    pages = np.arange(-(-length // PAGE)) if pages is None else np.asarray(pages)
    k, v = read_tokens(cache[np.asarray(table_row)[pages]], lay)
    pos = (pages[:, None] * PAGE + np.arange(PAGE)).reshape(-1)
    ok = pos < length

    def flat(x):
        return x.transpose(1, 0, 2, 3).reshape(lay["n_kv_heads"], -1, lay["d"])[:, ok]

    return flat(k), flat(v), pos[ok]


def rotate(x, pos, theta: float) -> np.ndarray:
    """x [n][heads][d] rotated at its tokens' positions."""
    return O.apply_rope(np.asarray(x, np.float64), np.asarray(pos)[:, None], theta)


def quantise(x):
    """int8 codes and fp16 scales of x [...][d] (fp32 values), group by group."""
    x = np.asarray(x, np.float32)
    flat = x.reshape(-1, GROUP)
    codes = np.zeros(flat.shape, np.int64)
    scales = np.zeros(flat.shape[0])
    for i, g in enumerate(flat):
        s, q = O.quantize_group(g, 8)
        codes[i], scales[i] = q, float(s)
    return codes.reshape(x.shape), scales.reshape(x.shape[:-1] + (x.shape[-1] // GROUP,))


def attention(q, k, v, scale=None):
    """q [heads][d], k, v [n_kv_heads][tokens][d] -> (out [heads][d], lse [heads], weights
    [heads][tokens], scores); zeros and -inf without tokens."""
    q = np.asarray(q, np.float64)
    H, d = q.shape
    G = H // k.shape[0]
    scale = 1.0 / np.sqrt(d) if scale is None else scale
    kk, vv = np.repeat(k, G, 0), np.repeat(v, G, 0)
    s = np.einsum("hd,htd->ht", q, kk) * scale
    if s.shape[1] == 0:
        return np.zeros((H, d)), np.full(H, -np.inf), s, s
    m = s.max(1, keepdims=True)
    e = np.exp(s - m)
    l = e.sum(1, keepdims=True)
    p = e / l
    return np.einsum("ht,htd->hd", p, vv), (m + np.log(l))[:, 0], p, s


def page_scores(q, bounds):
    """Scores [n_kv_heads][pages] of bounds [pages][n_kv_heads][2][d] for queries q [heads][d]."""
    q = np.asarray(q, np.float64)
    Hkv = bounds.shape[1]
    qg = q.reshape(Hkv, -1, 1, q.shape[1])
    lo, hi = (bounds[:, :, i].transpose(1, 0, 2)[:, None] for i in (0, 1))
    return np.maximum(qg * lo, qg * hi).sum(-1).max(1)


def choose(scores, length: int, n_sel: int, keep_first: int, keep_last: int) -> np.ndarray:
    """Chosen pages of one (sequence, KV head), ascending, -1 behind them."""
    P = -(-length // PAGE)
    if P <= n_sel:
        pages = list(range(P))
    else:
        ends = list(range(keep_first)) + list(range(P - keep_last, P))
        rest = sorted(range(keep_first, P - keep_last), key=lambda i: (-scores[i], i))
        pages = sorted(ends + rest[:n_sel - len(ends)])
    return np.array(pages + [-1] * (n_sel - len(pages)), np.int64)
