"""Cross attention with more queries than keys where a request has up to 16
(query, head) rows a kv head, which go to the split-KV decode: the queries'
positions L - Q + i are negative there."""
import pytest

from _shared import CrossRun, compare
from int8_kv_cache_reshape_gb300 import workloads as W

pytestmark = pytest.mark.gpu

DTYPES = ["auto", "fp8_e4m3", "fp8_e5m2", "int8_per_token_head", "fp8_per_token_head",
          "fp8_e5m2_per_token_head", "int4_per_token_head"]


@pytest.mark.parametrize("options", [{}, {"soft_cap": 20.0}])
@pytest.mark.parametrize("warps", [None, 4, 40])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("D", [64, 128, 256])
def test_more_queries_than_keys(cuda_device, monkeypatch, options, warps, dtype, D):
    """Tiles of 8 rows and of 16 a kv head, beside requests that are cut among
    warps, with sinks and without keys."""
    if warps:
        monkeypatch.setenv("KVQ_DECODE_WARPS", str(warps))
    new = [4, 8, 3, 8, 5, 4, 2, 8, 1, 6]
    lens = [1, 3, 2, 7, 4, 0, 300, 250, 1, 5]
    wl = W.custom("cross", new, lens, 4, 2, D, 16, dtype, 70 + D, causal=False, extra_blocks=2,
                  token_scale_range=(0.2, 5.0) if "per_token" in dtype else None, **options)
    g = CrossRun(wl, sinks=None if options else W.sink_logits(4, 5)).write_cache().attention()
    assert g.rect["num_units"] == 0 and g.sched_info["num_prefill_tiles"] == 0
    compare(g, f"{dtype} {D}")


@pytest.mark.parametrize("dtype", DTYPES)
def test_one_head_a_kv_head(cuda_device, dtype):
    """Sixteen queries of a group of one head to fifteen keys and fewer."""
    wl = W.custom("cross", [16, 9, 16, 2], [15, 8, 1, 1], 3, 3, 128, 16, dtype, 71, causal=False,
                  token_scale_range=(0.2, 5.0) if "per_token" in dtype else None)
    g = CrossRun(wl).write_cache().attention()
    assert g.rect["num_units"] == 0
    compare(g, dtype)
