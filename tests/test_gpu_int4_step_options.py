"""The 4-bit fused step with its options (window, soft cap, ALiBi, sinks), on
whole and cut tiles, in every instance of the kernel, from device and host
buffers, captured; and requests that the step leaves out.  Caches bit-exact
against the oracle, outputs within the bound of tests/_harness.py.
"""
import numpy as np
import pytest
import torch

from int8_kv_cache_reshape_gb300 import workloads as W

from _harness import assert_attention_close, kvq, oracle_cache, oracle_reference
from test_gpu_decode_step import Step
from test_gpu_int4_serving import _host_parts

pytestmark = pytest.mark.gpu

DT = "int4_per_token_head"

# whole tiles (one or two chunks of 32 tokens) beside tiles cut many times;
# lengths on and off the chunk's and the window's borders
LENS = [1, 33, 3000, 64, 700, 2049, 90]

# window, soft cap, ALiBi, sinks
OPTIONS = [(1, 0.0, False, False), (37, 0.0, False, False), (600, 20.0, False, False), (0, 5.0, False, False),
           (0, 0.0, True, False), (0, 0.0, False, True), (130, 0.0, True, False), (130, 30.0, True, True),
           (0, 30.0, True, True), (64, 0.0, False, True), (100000, 0.0, True, True)]


def _wl(D, hq, hkv, ql, window, cap, seed, lens=None, **kw):
    lens = [max(a, b) for a, b in zip(lens or LENS, ql)]
    return W.custom(f"int4-step-options-{D}-{hq}/{hkv}", ql, lens, hq, hkv, D, 16, DT, seed, window=window,
                    soft_cap=cap, token_scale_range=(0.1, 10.0), **kw)


def _extras(hq, alibi, sinks, seed=3):
    return (W.alibi_slopes(hq) if alibi else None, W.sink_logits(hq, seed) if sinks else None)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("hq,hkv,q", [(32, 8, 1), (16, 4, 4), (10, 2, 3)])
@pytest.mark.parametrize("window,cap,alibi,sinks", OPTIONS)
def test_options(cuda_device, D, hq, hkv, q, window, cap, alibi, sinks):
    rng = np.random.default_rng(D + q)
    ql = [int(x) for x in rng.integers(1, q + 1, len(LENS))]
    ql[2] = q
    wl = _wl(D, hq, hkv, ql, window, cap, 950 + D + q)
    Step(wl, *_extras(hq, alibi, sinks)).run().check(f"{wl.name} w{window} c{cap} a{alibi} s{sinks}")


@pytest.mark.parametrize("hkv", [1, 3, 13, 17, 24])
def test_options_with_split_heads(cuda_device, hkv):
    """Head counts that take one copy group, several, or one head each."""
    for D in (64, 128, 256):
        wl = _wl(D, 2 * hkv, hkv, [1, 2, 1], 200, 15.0, 970 + hkv, lens=[40, 900, 333])
        Step(wl, *_extras(2 * hkv, True, True)).run().check(f"{wl.name}")


@pytest.mark.parametrize("R", [256, 257, 400])
def test_options_of_many_requests(cuda_device, R):
    """Plans of every CTA's own and the first CTA's for all, windows cutting
    most requests."""
    rng = np.random.default_rng(R)
    wl = _wl(64, 8, 2, [1] * R, 50, 0.0, 980, lens=[int(x) for x in rng.integers(1, 150, R)])
    Step(wl, *_extras(8, True, True)).run().check(f"{R} requests")


def test_sinks_large_and_none(cuda_device):
    """A sink that takes nearly all the weight, one that takes none (-inf),
    one far below the scores."""
    wl = _wl(128, 8, 2, [1, 2, 1, 1, 1, 1, 1], 0, 0.0, 990)
    sinks = np.array([30.0, -np.inf, -80.0, 0.0, 12.0, -np.inf, 5.0, 60.0], np.float32)
    Step(wl, None, sinks).run().check("sinks")


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("alibi", [False, True])
def test_blocks_freed_behind_the_window(cuda_device, D, alibi):
    """A loop with a window frees the blocks behind it: their table entries
    (-1, or ids of blocks that hold NaN scales) are never read."""
    window = 100
    wl = _wl(D, 8, 2, [1, 2, 1, 1, 2, 1, 1], window, 0.0, 1000)
    a = Step(wl, *_extras(8, alibi, True)).run()
    a.check("all blocks")
    for entry in (-1, None):
        b = Step(wl, *_extras(8, alibi, True))
        for r, (L, Q) in enumerate(zip(wl.seq_lens, wl.query_lens)):
            gone = max(0, L - Q - window + 1) // 16
            if entry is None:
                blocks = wl.block_table[r, :gone].long().to(b.g.dev)
                b.g.kc[blocks] = 0xFF
                b.g.vc[blocks] = 0xFF
            else:
                b.g.bt[r, :gone] = entry
        b.run()
        torch.cuda.synchronize()
        kvq().decode_step_check(b.ws.t)
        assert torch.equal(b.g.out.view(torch.int16), a.g.out.view(torch.int16))


@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("alibi", [False, True])
def test_options_from_host_buffers(cuda_device, graph, alibi):
    wl = _wl(128, 32, 8, [1, 2, 1, 3, 1, 1, 2], 300, 25.0, 1010)
    extra = _extras(32, alibi, True)
    ref = Step(wl, *extra).run()
    ref.check("device inputs")
    want = ref.g.out.view(torch.int16).cpu()
    st = Step(wl, *extra)
    g = st.g
    h_in, d_in, (q, nk, nv, ns, qsl, sl, bt) = _host_parts(st)
    h_out = torch.full(g.out.shape, float("nan"), dtype=torch.bfloat16).pin_memory()
    make = kvq().decode_step_graph if graph else kvq().prepare_decode_step_host_io
    call = make(h_in, d_in, h_out, 0, nk, nv, ns, g.kc, g.vc, q, qsl, sl, bt, st.mql, wl.sm_scale, wl.window,
                wl.soft_cap, 1.0, 1.0, None, st.ws.t, DT, wl.heads_kv, alibi_slopes=g.alibi, sinks=g.sinks)
    for _ in range(2):
        h_out.fill_(float("nan"))
        torch.cuda.synchronize()
        call()
        torch.cuda.synchronize()
        assert torch.equal(h_out.view(torch.int16), want)
        assert torch.equal(g.kc, ref.g.kc) and torch.equal(g.vc, ref.g.vc)
    kvq().decode_step_check(st.ws.t)
    if graph:
        call.close()


def test_requests_without_new_tokens(cuda_device):
    wl = W.custom("int4-step-idle", [1, 0, 2, 0, 1], [500, 90, 40, 0, 1200], 16, 4, 128, 16, DT, 1020, window=77,
                  token_scale_range=(0.1, 10.0))
    Step(wl, *_extras(16, True, True)).run().check(wl.name)


@pytest.mark.parametrize("R", [3, 300])
def test_device_lengths_beyond_the_bound(cuda_device, R):
    """More new tokens than max_query_len on the device: the request is left
    out and flagged, its output rows stay; the others are right."""
    ql, lens = [1, 3, 1] + [1] * (R - 3), [500, 90, 40] + [20] * (R - 3)
    wl = W.custom("int4-step-bad", ql, lens, 16, 4, 128, 16, DT, 1030)
    st = Step(wl, max_query_len=2).run()
    torch.cuda.synchronize()
    with pytest.raises(kvq().KvqError) as e:
        kvq().decode_step_check(st.ws.t)
    assert e.value.status == kvq().E_INVALID_ARG
    kc, vc = oracle_cache(wl)
    toks = [0] + list(range(4, R + 2))
    ref, bnd = oracle_reference(wl, kc, vc, tokens=toks)
    assert_attention_close(st.g.out_f32(toks), ref, "4-bit step: good requests", bnd)
    assert torch.isnan(st.g.out[1:4].float()).all()
    # (the read cleared the word)
    kvq().decode_step_check(st.ws.t)


@pytest.mark.parametrize("block", [32, 48, 80, 2176])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_block_sizes(cuda_device, block, D):
    """Blocks that chunks of 32 tokens straddle, and one block a request."""
    wl = W.custom(f"int4-step-block-{block}", [1, 2, 1, 1], [1, 700, 97, 2048], 16, 4, D, block, DT, 1040 + D,
                  window=333, token_scale_range=(0.1, 10.0), extra_blocks=2)
    Step(wl, *_extras(16, False, True)).run().check(wl.name)
