"""Attention of decoder tokens to encoders' keys, against the oracle."""
import numpy as np
import pytest
import torch

from _harness import kvq
from _shared import CrossRun, compare
from int8_kv_cache_reshape_gb300 import workloads as W

pytestmark = pytest.mark.gpu

DTYPES = ["auto", "fp8_e4m3", "fp8_e5m2", "int8_per_token_head", "fp8_per_token_head",
          "fp8_e5m2_per_token_head", "int4_per_token_head"]


def _run(new, lens, Hq, Hkv, D, block, dtype, seed, alibi=None, sinks=None, **kw):
    wl = W.custom("cross", new, lens, Hq, Hkv, D, block, dtype, seed, causal=False, extra_blocks=2,
                  token_scale_range=(0.2, 5.0) if "per_token" in dtype else None, **kw)
    return CrossRun(wl, sinks=sinks).write_cache().attention()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("D,Hq,Hkv", [(64, 6, 6), (128, 8, 2), (256, 4, 1)])
def test_lengths(cuda_device, dtype, D, Hq, Hkv):
    """Single tokens, more tokens than keys, fewer, as many; no keys, no tokens."""
    new = [1, 1, 40, 200, 7, 33, 0, 1, 130, 3]
    lens = [90, 0, 9, 333, 7, 0, 50, 1, 1, 257]
    g = _run(new, lens, Hq, Hkv, D, 16, dtype, 50 + D)
    assert g.rect["num_units"] > 0
    compare(g, f"{dtype} {D}")


@pytest.mark.parametrize("dtype", DTYPES)
def test_options(cuda_device, dtype):
    g = _run([1, 50, 20, 4], [200, 150, 0, 333], 8, 2, 128, 16, dtype, 3, soft_cap=30.0, sinks=W.sink_logits(8, 5))
    compare(g, dtype)


@pytest.mark.parametrize("tiles", [1, 2, 100])
@pytest.mark.parametrize("group", [1, 3, 5, 7, 16])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_rows_and_cuts(cuda_device, monkeypatch, tiles, group, D):
    """Row tiles that begin inside a token's heads; keys cut into units of one,
    two and all KV tiles."""
    monkeypatch.setenv("KVQ_RECT_TILES", str(tiles))
    new = [1 + 17 // group, 128 // group + 1, 300 // group + 2, 40]
    g = _run(new, [300, 129, 64, 500], 2 * group, 2, D, 32, "int8_per_token_head", group)
    compare(g, f"group {group}, {tiles} tiles")


def test_the_decode_and_the_units_agree(cuda_device):
    """One batch of single tokens of 16 heads (decode) and of 17 rows (units)."""
    for new in (1, 2):
        compare(_run([new] * 5, [400, 33, 1, 128, 1000], 16, 1, 128, 16, "fp8_e4m3", 4), f"{new} tokens")


def test_static_scratch_and_refusals(cuda_device):
    k = kvq()
    g = _run([30, 2], [300, 77], 8, 2, 128, 16, "int8_per_token_head", 6)
    wl = g.wl
    sched = g.schedule()
    ws = torch.empty(max(256, sched.workspace_bytes), dtype=torch.uint8, device=cuda_device)
    args = lambda causal, window, **kw: dict(  # noqa: E731
        sched=sched, q=g.q, key_cache=g.kc, value_cache=g.vc, query_start_loc=g.qsl, seq_lens=g.sl, block_table=g.bt,
        sm_scale=wl.sm_scale, causal=causal, window=window, soft_cap=0.0, k_scale=1.0, v_scale=1.0, out=g.out,
        kv_cache_dtype=wl.kv_cache_dtype, heads_kv=2, **kw)
    want = g.out.clone()
    g.out.fill_(float("nan"))
    k.attention_with_kv_cache_static_scratch(**args(False, 0))
    torch.cuda.synchronize()
    assert torch.equal(g.out, want)
    slopes = torch.ones(8, device=cuda_device)
    for bad, status in ((dict(causal=True, window=0), k.E_SCHED_MISMATCH), (dict(causal=False, window=4), k.E_SCHED_MISMATCH),
                        (dict(causal=False, window=0, alibi_slopes=slopes), k.E_UNSUPPORTED)):
        with pytest.raises(k.KvqError) as e:
            k.attention_with_kv_cache(workspace=ws, **args(**bad))
        assert e.value.status == status
    with pytest.raises(k.KvqError) as e:
        k.attention_with_kv_cache(workspace=ws[:max(0, sched.workspace_bytes - 256)], **args(False, 0))
    assert e.value.status == k.E_WORKSPACE_TOO_SMALL
    sched.close()


def test_a_graph_replayed_on_other_encoders(cuda_device):
    """The keys of the cache change between replays; the lengths stay."""
    g = _run([5, 40, 1], [130, 260, 77], 8, 2, 128, 16, "int4_per_token_head", 6)
    wl, k = g.wl, kvq()
    sched = g.schedule()
    ws = torch.empty(max(256, sched.workspace_bytes), dtype=torch.uint8, device=cuda_device)
    graph = torch.cuda.CUDAGraph()

    def call():
        k.attention_with_kv_cache(sched, g.q, g.kc, g.vc, g.qsl, g.sl, g.bt, wl.sm_scale, False, 0, 0.0, 1.0, 1.0, g.out,
                                  ws, wl.kv_cache_dtype, 2)

    call()
    with torch.cuda.graph(graph):
        call()
    wl.key, wl.value = wl.value.clone(), wl.key.clone()
    g.key.copy_(wl.key)
    g.value.copy_(wl.value)
    g.write_cache()
    g.out.fill_(float("nan"))
    graph.replay()
    torch.cuda.synchronize()
    sched.check_device()
    compare(g, "replayed")
    sched.close()
