"""GPU parity of the 4-bit paged cache: the writer's bytes bit-exact against
the oracle, attention (decode rows, split tiles, prefill tiles, the fused
step) against the oracle's binary64 result within the bound of
tests/_harness.py.  That bound holds for 4-bit rows as it does for 8-bit
ones: a code times its group's multiplier enters the MMAs exactly, the row's
fp32 scale multiplies binary32 scores, and value scales join the softmax
weights before their one rounding to 11 bits.
"""
import numpy as np
import pytest
import torch

from int8_kv_cache_reshape_gb300 import workloads as W

from _harness import FILL, GpuRun, assert_attention_close, kvq, oracle_cache, oracle_reference
from test_gpu_decode_step import Step

pytestmark = pytest.mark.gpu

DT = "int4_per_token_head"


def _run(wl, tokens=None, **kw):
    g = GpuRun(wl, **kw).write_cache()
    kc, vc = oracle_cache(wl)
    assert np.array_equal(g.kc.cpu().numpy(), kc)
    assert np.array_equal(g.vc.cpu().numpy(), vc)
    g.attention()
    ref, bnd = oracle_reference(wl, kc, vc, tokens=tokens, **kw)
    return assert_attention_close(g.out_f32(tokens), ref, wl.name, bnd), g


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("hkv", [1, 3])
def test_cache_bytes(cuda_device, D, hkv):
    wl = W.custom("int4-cache", [1, 3, 1], [37, 50, 16], 2 * hkv, hkv, D, 16, DT, 100 + D, extra_blocks=3,
                  outlier_p=0.02, outlier_mul=40.0, token_scale_range=(1e-3, 1e3))
    wl.key[3] = 0                                  # a zero row
    wl.value[4, :, : D // 8] = 0                   # a zero group
    wl.key[5] = 1.0e-39                            # subnormals
    wl.value[6] = 3.0e38
    wl.key[8] = 7.0                                # quotients next to .5
    wl.key[8, 0, :6] = torch.tensor([0.5, 1.5, 2.5, -3.5, -0.5, 6.5])
    wl.slot_mapping[[0, 9, 40]] = -1
    wl.slot_mapping[7] = wl.num_blocks * wl.block_size + 3
    g = GpuRun(wl).write_cache()
    kc, vc = oracle_cache(wl)
    assert np.array_equal(g.kc.cpu().numpy(), kc)
    assert np.array_equal(g.vc.cpu().numpy(), vc)
    assert np.any(kc == FILL)


def test_cache_bytes_of_many_values(cuda_device):
    """Rows of every bf16 exponent and mantissa beside one another."""
    bits = np.arange(65536, dtype=np.uint32)
    pats = bits[((bits >> 7) & 0xFF) != 0xFF].astype(np.uint16)
    rng = np.random.default_rng(3)
    D, H = 128, 2
    x = np.concatenate([pats, rng.permutation(pats)])
    T = x.size // (H * D)
    x = torch.from_numpy(x[: T * H * D].copy().view(np.int16)).view(torch.bfloat16).view(T, H, D)
    wl = W.custom("int4-sweep", [1], [T], 2, H, D, 16, DT, 7)
    wl.key, wl.value = x, x.flip(0).contiguous()
    g = GpuRun(wl).write_cache()
    kc, vc = oracle_cache(wl)
    assert np.array_equal(g.kc.cpu().numpy(), kc)
    assert np.array_equal(g.vc.cpu().numpy(), vc)


@pytest.mark.parametrize("D,hq,hkv", [(64, 8, 8), (64, 8, 1), (128, 16, 8), (128, 12, 3), (256, 16, 2),
                                      (128, 16, 1), (256, 7, 1)])
def test_decode_shapes(cuda_device, D, hq, hkv):
    _run(W.custom(f"int4-{D}-{hq}/{hkv}", [1, 2, 1, 5, 1], [1, 17, 100, 5, 333], hq, hkv, D, 16, DT, 200 + D + hq,
                  outlier_p=0.01, token_scale_range=(0.1, 10.0)))


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("window,soft_cap", [(1, 0.0), (37, 30.0), (0, 5.0), (1000, 0.0)])
def test_window_and_soft_cap(cuda_device, D, window, soft_cap):
    _run(W.custom("int4-win", [1, 3, 1, 2], [700, 90, 16, 256], 16, 4, D, 32, DT, 300, window=window,
                  soft_cap=soft_cap))


@pytest.mark.parametrize("warps", [4, 12, 400, 100000])
def test_forced_warp_counts(cuda_device, monkeypatch, warps):
    monkeypatch.setenv("KVQ_DECODE_WARPS", str(warps))
    _run(W.custom("int4-splits", [1, 1, 2, 1], [1000, 129, 300, 16], 32, 8, 128, 16, DT, 302,
                  token_scale_range=(0.1, 10.0)))


@pytest.mark.parametrize("D,hq,hkv,block", [(64, 8, 2, 16), (128, 16, 4, 16), (128, 20, 4, 48), (256, 16, 2, 2176)])
def test_prefill(cuda_device, D, hq, hkv, block):
    ql = [70, 200, 33, 1]
    _run(W.custom(f"int4-prefill-{D}", ql, [70, 230, 300, 77], hq, hkv, D, block, DT, 400 + D,
                  outlier_p=0.01, token_scale_range=(0.1, 10.0)))


@pytest.mark.parametrize("D", [64, 128, 256])
def test_prefill_and_decode_options(cuda_device, D):
    hq = 16
    wl = W.custom("int4-ext", [90, 1, 140], [500, 777, 140], hq, 4, D, 16, DT, 410, window=130, soft_cap=20.0)
    _run(wl, alibi_slopes=W.alibi_slopes(hq), sinks=W.sink_logits(hq, 5))


def test_non_causal(cuda_device):
    _run(W.custom("int4-noncausal", [4, 1, 40], [60, 30, 90], 16, 4, 128, 16, DT, 301, causal=False))


def test_persistent_prefill_on_few_ctas(cuda_device, monkeypatch):
    """The same bits whichever CTA takes a tile."""
    wl = W.custom("int4-few", [150, 300, 20], [150, 500, 900], 16, 4, 128, 16, DT, 420, token_scale_range=(0.1, 10.0))
    _, a = _run(wl)
    for n in (1, 3):
        monkeypatch.setenv("KVQ_PREFILL_CTAS", str(n))
        b = GpuRun(wl).write_cache().attention()
        assert torch.equal(a.out.view(torch.int16), b.out.view(torch.int16))


@pytest.mark.parametrize("D,hq,hkv,ql", [(64, 10, 2, [3, 1, 2]), (128, 32, 8, [1] * 9), (256, 16, 1, [1, 1])])
def test_fused_step(cuda_device, D, hq, hkv, ql):
    rng = np.random.default_rng(len(ql) + D)
    sl = [int(x) for x in rng.integers(max(ql), 3000, len(ql))]
    sl[0] = ql[0]
    Step(W.custom(f"int4-step-{D}", ql, sl, hq, hkv, D, 16, DT, 600 + D, token_scale_range=(0.1, 10.0))).run().check(
        "int4 step")


@pytest.mark.parametrize("dtype", [DT, "int8_per_token_head", "fp8_per_token_head"])
@pytest.mark.parametrize("Q", [1, 40])
def test_zero_value_rows_at_the_start(cuda_device, dtype, Q):
    """Value rows whose scale is zero, from the first chunk (and the first
    KV tile) on: zeros weigh in, nothing turns into NaN.  One request has no
    other values: its output is zero."""
    wl = W.custom("zero-v", [Q, Q], [400, 200], 8, 2, 128, 16, dtype, 430)
    off = wl.seq_lens[0]
    wl.value[:150] = 0
    wl.value[off:] = 0
    wl.key[:20] = 0
    _, g = _run(wl)
    assert (g.out[Q:].float() == 0).all()


def test_hole_in_the_table(cuda_device):
    """Blocks outside the pool read as masked keys: the first block, one in
    the middle, and all of a request's (zero rows)."""
    for Q in (1, 30):
        wl = W.custom("int4-holes", [Q, Q], [200, 64], 8, 2, 128, 16, DT, 440, causal=False)
        g = GpuRun(wl).write_cache()
        g.bt[0, 0] = -1
        g.bt[0, 5] = wl.num_blocks + 3
        g.bt[1, :] = -1
        g.attention()
        # the oracle on the remaining keys: a table and lengths without the holes
        keep = [i for i in range(13) if i not in (0, 5)]
        kc, vc = oracle_cache(wl)
        wl2 = W.custom("int4-holes", [Q, Q], [200 - 32, 64], 8, 2, 128, 16, DT, 440, causal=False)
        wl2.q = wl.q
        wl2.num_blocks = wl.num_blocks
        bt = wl.block_table.clone()
        bt[0, : len(keep)] = wl.block_table[0, keep]
        wl2.block_table = bt
        ref, bnd = oracle_reference(wl2, kc, vc, tokens=range(Q))
        assert_attention_close(g.out_f32(range(Q)), ref, "int4 holes", bnd)
        assert (g.out[Q:].float() == 0).all()


def test_strided_rows_and_prepared_calls(cuda_device):
    """K and V as views of a fused projection's output (a token stride above
    Hkv * D), through the prepared calls, twice: the same bytes and bits."""
    k = kvq()
    wl = W.custom("int4-strided", [1, 1, 20], [300, 45, 100], 8, 2, 128, 16, DT, 450)
    g = GpuRun(wl)
    qkv = torch.zeros((wl.num_tokens, 12, 128), dtype=torch.bfloat16, device=g.dev)
    qkv[:, 8:10], qkv[:, 10:] = g.key, g.value
    write = k.prepare_reshape_and_cache(qkv[:, 8:10], qkv[:, 10:], g.kc, g.vc, g.slots, DT)
    sched = k.get_scheduler_metadata(3, 8, 2, 128, wl.seq_lens_t.numpy(), wl.query_start_loc.numpy(), True, 0, DT)
    ws = torch.empty(max(1, sched.workspace_bytes), dtype=torch.uint8, device=g.dev)
    attend = k.prepare_attention_with_kv_cache(sched, g.q, g.kc, g.vc, g.qsl, g.sl, g.bt, wl.sm_scale, True, 0, 0.0,
                                               1.0, 1.0, g.out, ws, DT, 2)
    outs = []
    for _ in range(2):
        write()
        attend()
        outs.append(g.out.clone())
    torch.cuda.synchronize()
    sched.check_device()
    kc, vc = oracle_cache(wl)
    assert np.array_equal(g.kc.cpu().numpy(), kc) and np.array_equal(g.vc.cpu().numpy(), vc)
    assert torch.equal(outs[0].view(torch.int16), outs[1].view(torch.int16))
    ref, bnd = oracle_reference(wl, kc, vc)
    assert_attention_close(g.out_f32(), ref, "int4 strided", bnd)
