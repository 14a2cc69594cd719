"""Score scales of zero and below: sm_scale is any finite number.  A negative
one prefers the keys that point away from the query, zero weighs all visible
keys alike.  Prefill and decode rows (masked and whole KV tiles, cut tiles),
every dtype, plain, capped and with ALiBi and sinks, and the fused step;
against the oracle within the bound of tests/_harness.py.
"""
import numpy as np
import pytest

from int8_kv_cache_reshape_gb300 import workloads as W

from _harness import ORACLE_DT, GpuRun, assert_attention_close, oracle_cache, oracle_reference
from test_gpu_decode_step import Step

pytestmark = pytest.mark.gpu

OPTIONS = [dict(), dict(window=70), dict(soft_cap=4.0), dict(extras=True), dict(causal=False)]


def _wl(dtype, D, scale, ql, sl, window=0, soft_cap=0.0, causal=True, **_):
    return W.custom(f"scale-{dtype}-{D}-{scale}", ql, sl, 8, 2, D, 16, dtype, 1200 + D, window=window,
                    soft_cap=soft_cap, causal=causal, sm_scale=scale)


def _extras(opt):
    return dict(alibi_slopes=W.alibi_slopes(8), sinks=W.sink_logits(8, 4)) if opt.get("extras") else {}


@pytest.mark.parametrize("dtype", list(ORACLE_DT))
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("scale", [-0.125, 0.0, -2.0])
@pytest.mark.parametrize("opt", range(len(OPTIONS)))
def test_attention(cuda_device, dtype, D, scale, opt):
    wl = _wl(dtype, D, scale, [90, 1, 2, 150], [330, 1500, 33, 150], **OPTIONS[opt])
    kw = _extras(OPTIONS[opt])
    g = GpuRun(wl, **kw).write_cache().attention()
    assert g.sched_info["num_prefill_tiles"] > 0 and g.sched_info["num_tiles"] > 0
    kc, vc = oracle_cache(wl)
    toks = list(range(0, 90, 7)) + [89, 90, 91, 92] + list(range(93, 243, 11)) + [242]
    ref, bnd = oracle_reference(wl, kc, vc, tokens=toks, **kw)
    assert_attention_close(g.out_f32(toks), ref, f"{wl.name} {opt}", bnd)
    if scale == 0.0 and opt == 0:
        # the mean of the values
        out = g.out_f32([90])[0, 0]
        assert np.abs(out).max() < 0.5


@pytest.mark.parametrize("dtype", ["int4_per_token_head", "int8_per_token_head", "fp8_e4m3", "auto"])
@pytest.mark.parametrize("scale", [-0.125, 0.0])
@pytest.mark.parametrize("opt", [0, 2, 3])
def test_step(cuda_device, dtype, scale, opt):
    wl = _wl(dtype, 128, scale, [1, 2, 1], [900, 40, 3000], **OPTIONS[opt])
    kw = _extras(OPTIONS[opt])
    Step(wl, kw.get("alibi_slopes"), kw.get("sinks")).run().check(f"{wl.name} {opt}")
