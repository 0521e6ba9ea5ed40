"""Numbers that the plain cache's calls would take for others are refused by the binding (no GPU)."""
import pytest
import torch

from rank_quantized_kv_decode_b200 import api


@pytest.fixture(scope="module")
def args():
    from rank_quantized_kv_decode_b200 import build
    build.build()
    lay = api.kv_layout_init(api.make_kv_config(8, 2, 64, "bf16", 10000.0))
    q = torch.zeros(2, 8, 64, dtype=torch.bfloat16)
    raw, i32 = torch.zeros(1 << 16, dtype=torch.uint8), torch.zeros(2, dtype=torch.int32)
    return lay, q, raw, torch.zeros(2, 4, dtype=torch.int32), i32


@pytest.mark.parametrize("kw,match", [
    (dict(window=(1 << 32) + 5), "window: 4294967301 does not fit"), (dict(window=1 << 32), "window: "),
    (dict(window=1 << 31), "window: "), (dict(max_ctas=(1 << 32) + 1), "max_ctas: "), (dict(window=-(1 << 31) - 1), "window: "),
    (dict(scale=1e-50), "scale: 1e-50 is 0 in fp32"), (dict(scale=-1e-60), "scale: ")])
def test_decode(args, kw, match):
    lay, q, raw, table, i32 = args
    with pytest.raises(ValueError, match=match):
        api.kv_decode(lay, q, raw, table, i32, q.clone(), raw, i32, **kw)


@pytest.mark.parametrize("kw", [dict(keep_first=1 << 32), dict(keep_last=(1 << 32) + 1), dict(keep_first=-(1 << 40))])
def test_select(args, kw):
    lay, q, raw, table, i32 = args
    with pytest.raises(ValueError, match=f"{next(iter(kw))}: .* does not fit in 32 bits"):
        api.kv_select(lay, q, raw, table, i32, torch.zeros(2, 2, 3, dtype=torch.int32), i32, **kw)


def test_the_largest_that_fit_reach_the_other_checks(args):
    lay, q, raw, table, i32 = args
    with pytest.raises(ValueError, match="CUDA tensor"):
        api.kv_decode(lay, q, raw, table, i32, q.clone(), raw, i32, window=(1 << 31) - 1, scale=1e-40)
