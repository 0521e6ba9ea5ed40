"""Host-side checks of the plain key-value cache (no GPU): layout and sizes against the oracle's own
layout, refusals of the entry points and of the binding before anything touches a device, and
the oracle's pieces on cases worked out by hand."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest
import torch

from oracle import kv_oracle as K
from rank_quantized_kv_decode_b200 import _lib as L
from rank_quantized_kv_decode_b200 import api


@pytest.fixture(scope="module")
def lib():
    from rank_quantized_kv_decode_b200 import build
    build.build()
    return L.load()


def layout(fmt="bf16", H=8, Hkv=2, d=128):
    return api.kv_layout_init(api.make_kv_config(H, Hkv, d, fmt, 10000.0))


@pytest.mark.parametrize("fmt", ["bf16", "f16", "int8"])
@pytest.mark.parametrize("H,Hkv,d", [(32, 8, 128), (4, 4, 64), (10, 2, 128), (64, 1, 64)])
def test_layout_matches_oracle(lib, fmt, H, Hkv, d):
    lay, want = layout(fmt, H, Hkv, d), K.kv_page_layout(fmt, Hkv, d)
    for f in ("page_bytes", "token_bytes", "off_heads", "head_bytes", "off_v", "off_ks", "off_vs"):
        assert getattr(lay, f) == want[f], f
    assert lay.page_bytes % 16 == 0 and lay.head_bytes % 16 == 0


def test_struct_sizes(lib):
    assert ctypes.sizeof(L.KvConfig) == 32
    assert ctypes.sizeof(L.KvLayout) == 32 + 7 * 8
    assert ctypes.sizeof(L.KvDecodeOpts) == 16


def test_alloc_sizes(lib):
    lay = layout()
    s = api.kv_alloc(lay, 7, 3, 70)
    assert s.cache_bytes == 7 * lay.page_bytes
    # the table of the latent cache at the same head_dim and length
    assert s.rope_table_bytes == (128 + 35) * 64 * 8
    # a record of four heads for each piece: nine chunks for each of 296 x 4 warps (d 64: 444 x 4), and one more where
    # each of 3 x 2 (sequence, KV head) ends; a counter before them
    assert s.decode_workspace_bytes == 256 + (296 * 4 * 9 + 3 * 2) * 4 * (128 * 4 + 8)
    # twenty query heads per KV head: three groups of at most eight
    s = api.kv_alloc(layout("bf16", 40, 2, 64), 1, 5, 32)
    assert s.decode_workspace_bytes == 256 + (444 * 4 * 9 + 5 * 2 * 3) * 8 * (64 * 4 + 8)
    for args in ((-1, 1, 1), (1, 1, 0), (1, 1, (1 << 24) + 1), (1 << 62, 1, 1), (1, -1, 1), (1, 65536, 1),
                 (1, 65535, 1 << 13)):
        with pytest.raises(L.StarkvError) as e:
            api.kv_alloc(lay, *args)
        assert e.value.status == L.ERR_INVALID_ARG


@pytest.mark.parametrize("field,value,status", [
    ("n_kv_heads", 0, L.ERR_INVALID_ARG), ("n_kv_heads", 65, L.ERR_INVALID_ARG),
    ("n_q_heads", 7, L.ERR_INVALID_ARG), ("n_q_heads", 0, L.ERR_INVALID_ARG),
    ("n_q_heads", 2 * 65, L.ERR_UNSUPPORTED), ("head_dim", 96, L.ERR_UNSUPPORTED),
    ("fmt", 3, L.ERR_INVALID_ARG), ("fmt", -1, L.ERR_INVALID_ARG), ("page_tokens", 32, L.ERR_UNSUPPORTED),
    ("reserved", 1, L.ERR_INVALID_ARG), ("rope_theta", 1.0, L.ERR_INVALID_ARG),
    ("rope_theta", float("nan"), L.ERR_INVALID_ARG), ("rope_theta", float("inf"), L.ERR_INVALID_ARG)])
def test_layout_rejects(lib, field, value, status):
    cfg = api.make_kv_config(8, 2, 128, "bf16", 10000.0)
    setattr(cfg, field, value)
    with pytest.raises(L.StarkvError) as e:
        api.kv_layout_init(cfg)
    assert e.value.status == status


def test_tampered_layout_rejected(lib):
    lay = layout()
    lay.head_bytes += 16
    with pytest.raises(L.StarkvError) as e:
        api.kv_alloc(lay, 1, 1, 1)
    assert e.value.status == L.ERR_INVALID_ARG


# Addresses that no call may reach: every refusal below comes before the device is asked.
P16 = ctypes.c_void_p(0x10000)
ODD = ctypes.c_void_p(0x10008)


def append(lib, lay, q=P16, qs=1024, k=P16, ks=256, v=P16, vs=256, n=1, seq=P16, pos=P16, bt=P16, mp=2, batch=1,
           rope=P16, rb=1 << 30, cache=P16, pages=1, qo=P16, st=P16):
    return lib.starkv_kv_append(ctypes.byref(lay) if lay else None, q, qs, k, ks, v, vs, n, seq, pos, bt, mp, batch,
                                rope, rb, cache, pages, qo, st, None)


@pytest.mark.parametrize("kw,status", [
    (dict(n=-1), L.ERR_INVALID_ARG), (dict(n=(1 << 31) // 16), L.ERR_INVALID_ARG), (dict(batch=0), L.ERR_INVALID_ARG), (dict(mp=0), L.ERR_INVALID_ARG),
    (dict(mp=(1 << 24) + 1), L.ERR_INVALID_ARG), (dict(pages=0), L.ERR_INVALID_ARG),
    (dict(k=None), L.ERR_INVALID_ARG), (dict(v=None), L.ERR_INVALID_ARG), (dict(seq=None), L.ERR_INVALID_ARG),
    (dict(pos=None), L.ERR_INVALID_ARG), (dict(bt=None), L.ERR_INVALID_ARG), (dict(rope=None), L.ERR_INVALID_ARG),
    (dict(cache=None), L.ERR_INVALID_ARG), (dict(st=None), L.ERR_INVALID_ARG),
    (dict(qo=None), L.ERR_INVALID_ARG), (dict(q=None), L.ERR_INVALID_ARG),
    (dict(qs=1016), L.ERR_INVALID_ARG), (dict(qs=1028), L.ERR_INVALID_ARG), (dict(ks=248), L.ERR_INVALID_ARG),
    (dict(ks=260), L.ERR_INVALID_ARG), (dict(vs=-256), L.ERR_INVALID_ARG),
    (dict(qs=2048), L.ERR_INVALID_ARG),  # in place, but not contiguous
    (dict(q=ODD), L.ERR_INVALID_ARG), (dict(k=ODD), L.ERR_INVALID_ARG), (dict(v=ODD), L.ERR_INVALID_ARG),
    (dict(qo=ODD), L.ERR_INVALID_ARG), (dict(cache=ODD), L.ERR_INVALID_ARG), (dict(rope=ODD), L.ERR_INVALID_ARG),
    (dict(rb=8), L.ERR_WORKSPACE)])
def test_append_refuses_before_touching_the_device(lib, kw, status):
    assert append(lib, layout(), **kw) == status
    assert lib.starkv_last_error()


def test_append_of_nothing_is_ok_and_a_null_layout_is_not(lib):
    assert append(lib, layout(), n=0, k=None, cache=None) == L.OK
    assert append(lib, None) == L.ERR_INVALID_ARG


def decode(lib, lay, q=P16, cache=P16, pages=1, bt=P16, mp=2, lens=P16, batch=1, sel=None, n_sel=0, opts=None,
           out=P16, lse=None, ws=P16, wb=1 << 30, st=P16):
    o = ctypes.byref(L.KvDecodeOpts(*opts)) if opts else None
    return lib.starkv_kv_decode(ctypes.byref(lay), q, cache, pages, bt, mp, lens, batch, sel, n_sel, o, out, lse, ws,
                                wb, st, None)


@pytest.mark.parametrize("kw,status", [
    (dict(batch=-1), L.ERR_INVALID_ARG), (dict(batch=65536), L.ERR_INVALID_ARG), (dict(mp=0), L.ERR_INVALID_ARG),
    (dict(pages=0), L.ERR_INVALID_ARG), (dict(q=None), L.ERR_INVALID_ARG), (dict(cache=None), L.ERR_INVALID_ARG),
    (dict(bt=None), L.ERR_INVALID_ARG), (dict(lens=None), L.ERR_INVALID_ARG), (dict(out=None), L.ERR_INVALID_ARG),
    (dict(ws=None), L.ERR_INVALID_ARG), (dict(st=None), L.ERR_INVALID_ARG), (dict(q=ODD), L.ERR_INVALID_ARG),
    (dict(out=ODD), L.ERR_INVALID_ARG), (dict(cache=ODD), L.ERR_INVALID_ARG), (dict(ws=ODD), L.ERR_INVALID_ARG),
    (dict(sel=P16, n_sel=0), L.ERR_INVALID_ARG), (dict(sel=P16, n_sel=4, opts=(0.0, 64, 0, 0)), L.ERR_INVALID_ARG),
    (dict(opts=(-1.0, 0, 0, 0)), L.ERR_INVALID_ARG), (dict(opts=(float("nan"), 0, 0, 0)), L.ERR_INVALID_ARG),
    (dict(opts=(float("inf"), 0, 0, 0)), L.ERR_INVALID_ARG), (dict(opts=(3e38, 0, 0, 0)), L.ERR_INVALID_ARG), (dict(opts=(0.0, -1, 0, 0)), L.ERR_INVALID_ARG),
    (dict(opts=(0.0, 0, -1, 0)), L.ERR_INVALID_ARG), (dict(opts=(0.0, 0, 0, 1)), L.ERR_INVALID_ARG),
    (dict(wb=64), L.ERR_WORKSPACE)])
def test_decode_refuses_before_touching_the_device(lib, kw, status):
    assert decode(lib, layout(), **kw) == status


def test_decode_of_an_empty_batch_is_ok(lib):
    assert decode(lib, layout(), batch=0, q=None, out=None) == L.OK


def select(lib, lay, q=P16, cache=P16, pages=1, bt=P16, mp=64, lens=P16, batch=1, n_sel=8, first=1, last=1, sel=P16,
           st=P16):
    return lib.starkv_kv_select(ctypes.byref(lay), q, cache, pages, bt, mp, lens, batch, n_sel, first, last, sel, st,
                                None)


@pytest.mark.parametrize("kw,status", [
    (dict(last=0), L.ERR_INVALID_ARG), (dict(first=-1), L.ERR_INVALID_ARG), (dict(n_sel=1), L.ERR_INVALID_ARG),
    (dict(n_sel=0, first=0), L.ERR_INVALID_ARG), (dict(first=2**31 - 1), L.ERR_INVALID_ARG),
    (dict(mp=L.KV_MAX_SELECT_PAGES + 1), L.ERR_UNSUPPORTED), (dict(batch=-1), L.ERR_INVALID_ARG),
    (dict(q=None), L.ERR_INVALID_ARG), (dict(sel=None), L.ERR_INVALID_ARG), (dict(lens=None), L.ERR_INVALID_ARG),
    (dict(q=ODD), L.ERR_INVALID_ARG), (dict(cache=ODD), L.ERR_INVALID_ARG), (dict(mp=0), L.ERR_INVALID_ARG)])
def test_select_refuses_before_touching_the_device(lib, kw, status):
    assert select(lib, layout(), **kw) == status


def test_binding_checks_types_and_shapes_before_the_library_sees_a_pointer(lib):
    lay = layout("bf16", 8, 2, 64)
    i32, table, raw = torch.zeros(4, dtype=torch.int32), torch.zeros(2, 4, dtype=torch.int32), torch.zeros(
        1 << 16, dtype=torch.uint8)
    k = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    q = torch.zeros(3, 8, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="k: expected dtype"):
        api.kv_append(lay, k.half(), k, i32, i32, table, raw, raw, i32)
    with pytest.raises(ValueError, match="k: expected shape"):
        api.kv_append(lay, k[:, :1], k, i32, i32, table, raw, raw, i32)
    with pytest.raises(ValueError, match="v: expected shape"):
        api.kv_append(lay, k, k[:2], i32, i32, table, raw, raw, i32)
    with pytest.raises(ValueError, match="heads of a token must be contiguous"):
        api.kv_append(lay, k.transpose(0, 1).contiguous().transpose(0, 1), k, i32, i32, table, raw, raw, i32)
    with pytest.raises(ValueError, match="tok_pos: 2 elements"):
        api.kv_append(lay, k, k, i32, i32[:2], table, raw, raw, i32)
    with pytest.raises(ValueError, match="q_out: "):
        api.kv_append(lay, k, k, i32, i32, table, raw, raw, i32, q=q, q_out=q[:1])
    with pytest.raises(ValueError, match="CUDA tensor"):
        api.kv_append(lay, k, k, i32, i32, table, raw, raw, i32)
    with pytest.raises(ValueError, match="k_out: "):
        api.kv_gather(lay, raw, i32, i32, table, k, k, i32)
    lens = i32[:2]
    out = torch.zeros(2, 8, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="q: 512 elements"):
        api.kv_decode(lay, q[:1], raw, table, lens, out, raw, i32)
    with pytest.raises(ValueError, match="out: expected dtype"):
        api.kv_decode(lay, q, raw, table, lens, out.float(), raw, i32)
    with pytest.raises(ValueError, match="lse: "):
        api.kv_decode(lay, q, raw, table, lens, out, raw, i32, lse=torch.zeros(8))
    with pytest.raises(ValueError, match="block_table: 1 rows for 2 sequences"):
        api.kv_decode(lay, q, raw, table[:1], lens, out, raw, i32)
    sel = torch.zeros(2, 2, 3, dtype=torch.int32)
    with pytest.raises(ValueError, match="sel: expected"):
        api.kv_decode(lay, q, raw, table, lens, out, raw, i32, sel=sel[:, :1])
    with pytest.raises(ValueError, match="sel: expected 3 dimensions"):
        api.kv_select(lay, q, raw, table, lens, sel[0], i32)
    with pytest.raises(ValueError, match="CUDA tensor"):
        api.kv_decode(lay, q, raw, table, lens, out, raw, i32, sel=sel)


def test_oracle_bound_is_attained_at_a_corner_and_never_passed():
    r = np.random.default_rng(1)
    k, q = r.standard_normal((3, 2, 64, 8)), r.standard_normal((4, 8))
    bounds = np.stack((k.min(2), k.max(2)), 2)
    s = K.page_scores(q, bounds)
    dots = np.einsum("ghd,pgtd->gpht", q.reshape(2, 2, 8), k).max((2, 3))
    assert np.all(s >= dots - 1e-12)
    # one channel: the bound is the larger of two products
    b = np.array([[[[-2.0], [3.0]]]])
    assert K.page_scores(np.array([[-5.0]]), b)[0, 0] == 10.0
    assert K.page_scores(np.array([[5.0]]), b)[0, 0] == 15.0


def test_oracle_choice_by_hand():
    scores = np.array([9.0, 1.0, 7.0, 7.0, 7.0, 2.0, 0.0])
    # 7 pages, 4 wanted: the last, and of the rest 9, 7 and 7 (the lower pages of the three equal ones)
    assert list(K.choose(scores, 7 * 64, 4, 0, 1)) == [0, 2, 3, 6]
    assert list(K.choose(scores, 7 * 64 - 63, 5, 2, 2)) == [0, 1, 2, 5, 6]
    assert list(K.choose(scores, 3 * 64, 4, 0, 1)) == [0, 1, 2, -1]
    assert list(K.choose(scores, 0, 2, 0, 1)) == [-1, -1]


def test_oracle_attention_by_hand():
    # equal scores: the mean of the values; ln 2 + score
    k = np.ones((1, 2, 4))
    v = np.array([[[1.0, 2, 3, 4], [3.0, 4, 5, 6]]])
    o, lse, _, _ = K.attention(np.ones((2, 4)), k, v)
    assert np.allclose(o, [[2, 3, 4, 5]] * 2) and np.allclose(lse, 2.0 + np.log(2.0))


C_PROGRAM = r"""
#include <stdio.h>
#include <string.h>
#include "starkv.h"

int main(void) {
  starkv_kv_config cfg;
  memset(&cfg, 0, sizeof cfg);
  cfg.n_q_heads = 32;
  cfg.n_kv_heads = 8;
  cfg.head_dim = 128;
  cfg.fmt = STARKV_KV_INT8;
  cfg.page_tokens = 64;
  cfg.rope_theta = 500000.0;
  starkv_kv_layout lay;
  starkv_kv_sizes sz;
  if (starkv_kv_layout_init(&cfg, &lay) != STARKV_OK) return 1;
  if (starkv_kv_alloc(&lay, 10, 4, 8, &sz) != STARKV_OK) return 2;
  /* refused before the device is touched */
  if (starkv_kv_append(&lay, NULL, 0, NULL, 0, NULL, 0, -1, NULL, NULL, NULL, 1, 1, NULL, 0, NULL, 1, NULL, NULL,
                       NULL) != STARKV_ERR_INVALID_ARG) return 3;
  if (starkv_kv_gather(&lay, NULL, 1, NULL, NULL, 0, NULL, 1, 1, NULL, NULL, NULL, NULL) != STARKV_OK) return 4;
  if (starkv_kv_select(&lay, NULL, NULL, 1, NULL, 1, NULL, 1, 4, 0, 0, NULL, NULL, NULL) != STARKV_ERR_INVALID_ARG) return 5;
  if (starkv_kv_decode(&lay, NULL, NULL, 1, NULL, 1, NULL, 0, NULL, 0, NULL, NULL, NULL, NULL, 0, NULL, NULL) !=
      STARKV_OK) return 6;
  printf("%lld %lld %lld\n", (long long)lay.page_bytes, (long long)lay.off_ks, (long long)sz.cache_bytes);
  return 0;
}
"""


@pytest.mark.skipif(shutil.which("gcc") is None, reason="no C compiler")
def test_c99_caller(lib, tmp_path):
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    libdir = os.path.join(root, "rank_quantized_kv_decode_b200")
    src, exe = tmp_path / "caller.c", tmp_path / "caller"
    src.write_text(C_PROGRAM)
    proc = subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-I", os.path.join(root, "include"), str(src), "-o",
                           str(exe), "-L", libdir, "-lstarkv", "-Wl,-rpath," + libdir,
                           "-Wl,--unresolved-symbols=ignore-in-shared-libs"], capture_output=True, text=True)
    assert proc.returncode == 0, proc.stderr
    run = subprocess.run([str(exe)], capture_output=True, text=True)
    assert run.returncode == 0, (run.returncode, run.stdout)
    want = K.kv_page_layout("int8", 8, 128)
    assert run.stdout.split() == [str(want["page_bytes"]), str(want["off_ks"]), str(10 * want["page_bytes"])]
