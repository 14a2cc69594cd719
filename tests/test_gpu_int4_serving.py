"""The 4-bit cache as a serving loop uses it: one call after another without
a synchronisation between them, on other streams, captured in CUDA graphs,
from host buffers; caches beyond 4 GiB; every split of the kv heads over the
decode's copy groups; NaN bit patterns in rows that no key holds.

The kernels of 4-bit rows are launched as programmatic dependents of what
runs before them on the stream, so each chain below is also a test that they
wait for it.
"""
import numpy as np
import pytest
import torch

from int8_kv_cache_reshape_gb300 import workloads as W

from _harness import GpuRun, assert_attention_close, kvq, oracle_cache, oracle_reference
from test_gpu_decode_step import Step, _pack_into

pytestmark = pytest.mark.gpu

DT = "int4_per_token_head"


def _bits(t):
    return t.view(torch.int16) if t.dtype == torch.bfloat16 else t


def _prepared(g, stream=None):
    """(schedule, workspace, write call, attention call) of a GpuRun."""
    wl, k = g.wl, kvq()
    s = k.get_scheduler_metadata(wl.num_req, wl.heads_q, wl.heads_kv, wl.head_dim, wl.seq_lens_t.numpy(),
                                 wl.query_start_loc.numpy(), wl.causal, wl.window, DT)
    ws = torch.zeros(max(s.workspace_bytes, 256), dtype=torch.uint8, device=g.dev)
    write = k.prepare_reshape_and_cache(g.key, g.value, g.kc, g.vc, g.slots, DT, stream=stream)
    attn = k.prepare_attention_with_kv_cache(
        s, g.q, g.kc, g.vc, g.qsl, g.sl, g.bt, wl.sm_scale, wl.causal, wl.window, wl.soft_cap, 1.0, 1.0, g.out,
        ws, DT, wl.heads_kv, stream=stream, alibi_slopes=g.alibi, sinks=g.sinks)
    return s, ws, write, attn


MIXED = dict(ql=[1, 90, 2, 1, 40], sl=[700, 300, 33, 1, 90])


def _mixed(seed, D=128, hq=16, hkv=4, **kw):
    return W.custom("int4-mixed", MIXED["ql"], MIXED["sl"], hq, hkv, D, 16, DT, seed,
                    token_scale_range=(0.1, 10.0), **kw)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_steps_one_after_another(cuda_device, D):
    """Inputs, lengths and tables rewritten on the stream right before each
    write + attention + read back: each gives what it gives alone."""
    runs = [_mixed(700 + i, D) for i in range(6)]
    g = GpuRun(_mixed(700, D, extra_blocks=0))
    s, ws, write, attn = _prepared(g)
    alone = []
    for wl in runs:
        a = GpuRun(wl).write_cache().attention()
        alone.append((a.out.clone(), a.kc.clone()))
    dev = g.dev
    src = [{n: t.to(dev) for n, t in (("q", w.q), ("key", w.key), ("value", w.value), ("slots", w.slot_mapping),
                                      ("bt", w.block_table))} for w in runs]
    qsl = g.qsl.clone()
    rows = torch.empty((sum(MIXED["sl"]), 4, D), dtype=torch.float32, device=dev)
    rows_v = torch.empty_like(rows)
    read = kvq().prepare_gather_cache(g.kc, g.vc, g.slots, rows, rows_v, DT)
    got = []
    torch.cuda.synchronize()
    for _ in range(3):
        got.clear()
        for x in src:
            g.out.fill_(float("nan"))
            g.qsl.zero_()                       # right only by the time the kernels may read it
            for n in ("q", "key", "value", "slots", "bt"):
                getattr(g, n).copy_(x[n])
            g.qsl.copy_(qsl)
            write()
            attn()
            read()
            got.append((g.out.clone(), rows.clone(), g.kc.clone()))
        torch.cuda.synchronize()
        s.check_device()
        for (out, r, kc), (want, want_kc), wl in zip(got, alone, runs):
            assert torch.equal(_bits(out), _bits(want))
            bt = wl.slot_mapping.to(dev)
            flat, want_flat = kc.flatten(0, 1)[bt], want_kc.flatten(0, 1)[bt]
            assert torch.equal(flat, want_flat)
    a = torch.empty_like(rows)
    b = torch.empty_like(rows)
    kvq().gather_cache(g.kc, g.vc, g.slots, a, b, DT)
    assert torch.equal(a, got[-1][1])


def test_captured_and_replayed(cuda_device):
    """Write, attention and read back captured in one graph; replays follow
    the inputs, also with another graph's replays between them."""
    k = kvq()
    runs = [_mixed(720), _mixed(721)]
    want = [GpuRun(w).write_cache().attention().out.clone() for w in runs]
    graphs = []
    for w in (runs[0], runs[0]):
        g = GpuRun(w)
        s, ws, write, attn = _prepared(g)
        rows, rows_v = (torch.empty(tuple(w.key.shape), dtype=torch.bfloat16, device=g.dev) for _ in range(2))
        side = torch.cuda.Stream()
        s2, ws2, write2, attn2 = _prepared(g, stream=side.cuda_stream)
        with torch.cuda.stream(side):
            write2(), attn2()                       # (the plan's upload stays out of the graph)
            torch.cuda.synchronize()
            gr = torch.cuda.CUDAGraph()
            with torch.cuda.graph(gr, stream=side):
                write2()
                attn2()
                k.gather_cache(g.kc, g.vc, g.slots, rows, rows_v, DT, stream=side.cuda_stream)
        graphs.append((g, gr, s2, ws2, rows, rows_v, s, ws))
    for i in (0, 1, 0):
        for (g, gr, *_), j in zip(graphs, (i, 1 - i)):
            w = runs[j]
            for n, t in (("q", w.q), ("key", w.key), ("value", w.value), ("slots", w.slot_mapping),
                         ("bt", w.block_table)):
                getattr(g, n).copy_(t.to(g.dev))
            g.out.fill_(float("nan"))
        for g, gr, *_ in graphs:
            gr.replay()
        torch.cuda.synchronize()
        for (g, gr, s2, *_), j in zip(graphs, (i, 1 - i)):
            s2.check_device()
            assert torch.equal(_bits(g.out), _bits(want[j]))


def test_two_streams(cuda_device):
    """Two steps of their own caches and workspaces at once."""
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    parts, want = [], []
    for i, st in enumerate(streams):
        w = _mixed(740 + i, (128, 64)[i])
        want.append(GpuRun(w).write_cache().attention().out.clone())
        g = GpuRun(w)
        parts.append((g,) + _prepared(g, stream=st.cuda_stream))
    torch.cuda.synchronize()
    for _ in range(20):
        for g, s, ws, write, attn in parts:
            write()
            attn()
    torch.cuda.synchronize()
    for (g, s, *_), o in zip(parts, want):
        s.check_device()
        assert torch.equal(_bits(g.out), _bits(o))


@pytest.mark.parametrize("D,hkv", [(64, 16), (64, 17), (64, 20), (64, 24), (64, 32), (64, 1), (128, 16), (128, 17),
                                   (128, 24), (128, 32), (128, 2), (256, 8), (256, 12), (256, 13), (256, 32),
                                   (256, 5)])
@pytest.mark.parametrize("G,Q", [(1, 2), (5, 3)])
def test_every_split_of_the_heads(cuda_device, D, hkv, G, Q):
    wl = W.custom(f"int4-heads-{D}-{hkv}", [1, Q, Q], [1, 95, 410], G * hkv, hkv, D, 16, DT, 760 + hkv,
                  token_scale_range=(0.1, 10.0))
    g = GpuRun(wl).write_cache()
    kc, vc = oracle_cache(wl)
    assert np.array_equal(g.kc.cpu().numpy(), kc)
    g.attention()
    ref, bnd = oracle_reference(wl, kc, vc)
    assert_attention_close(g.out_f32(), ref, wl.name, bnd)
    Step(wl).run().check("step " + wl.name)


@pytest.mark.parametrize("R", [256, 257, 700])
def test_step_of_many_requests(cuda_device, R):
    """Around the largest batch that every CTA plans for itself."""
    rng = np.random.default_rng(R)
    wl = W.custom(f"int4-many-{R}", [1] * R, [int(x) for x in rng.integers(1, 150, R)], 8, 2, 64, 16, DT, 780,
                  token_scale_range=(0.1, 10.0))
    Step(wl).run().check(wl.name)


def _host_parts(st):
    g = st.g
    parts = [g.q, st.nkey, st.nval, st.nslot, g.qsl, g.sl, g.bt]
    offs, o = [], 0
    for t in parts:
        offs.append(o)
        o += (t.numel() * t.element_size() + 255) // 256 * 256
    h_in = torch.zeros(o, dtype=torch.uint8).pin_memory()
    _pack_into(h_in, offs, parts)
    d_in = torch.full((o,), 0xA5, dtype=torch.uint8, device=g.dev)
    views = [d_in[off:off + t.numel() * t.element_size()].view(t.dtype).view(t.shape)
             for t, off in zip(parts, offs)]
    return h_in, d_in, views


@pytest.mark.parametrize("graph", [False, True])
def test_step_from_host_buffers(cuda_device, graph):
    wl = W.custom("int4-host-io", [1, 2, 1, 3, 1], [700, 333, 1, 2048, 96], 32, 8, 128, 16, DT, 790,
                  token_scale_range=(0.1, 10.0))
    ref = Step(wl).run()
    ref.check("device inputs")
    want = ref.g.out.view(torch.int16).cpu()
    st = Step(wl)
    g = st.g
    h_in, d_in, (q, nk, nv, ns, qsl, sl, bt) = _host_parts(st)
    h_out = torch.full(g.out.shape, float("nan"), dtype=torch.bfloat16).pin_memory()
    args = (nk, nv, ns, g.kc, g.vc, q, qsl, sl, bt, st.mql, wl.sm_scale, wl.window, wl.soft_cap, 1.0, 1.0, None,
            st.ws.t, DT, wl.heads_kv)
    call = (kvq().decode_step_graph if graph else kvq().prepare_decode_step_host_io)(h_in, d_in, h_out, 0, *args)
    for _ in range(3):
        h_out.fill_(float("nan"))
        d_in.fill_(0xA5)
        torch.cuda.synchronize()
        call()
        torch.cuda.synchronize()
        assert torch.equal(h_out.view(torch.int16), want)
        assert torch.equal(g.kc, ref.g.kc) and torch.equal(g.vc, ref.g.vc)
    kvq().decode_step_check(st.ws.t)
    if graph:
        call.close()


@pytest.mark.parametrize("Q", [1, 40])
def test_nan_bytes_in_rows_without_a_key(cuda_device, Q):
    """0xFF in every row that holds no key (scales read as NaN)."""
    wl = W.custom("int4-nan", [Q, 1, Q], [60, 17, 333], 16, 4, 128, 16, DT, 800, extra_blocks=4)
    a = GpuRun(wl).write_cache().attention()
    b = GpuRun(wl)
    b.kc.fill_(0xFF)
    b.vc.fill_(0xFF)
    kvq().reshape_and_cache(b.key, b.value, b.kc, b.vc, b.slots, DT)
    torch.cuda.synchronize()
    b.attention()
    assert not torch.isnan(b.out.float()).any()
    assert torch.equal(_bits(a.out), _bits(b.out))


@pytest.mark.parametrize("Q", [1, 33])
def test_cache_beyond_4_gib(cuda_device, Q):
    """The last blocks of caches of 4.6 GB each: the same rows and outputs as
    in small ones."""
    wl = W.custom("int4-far", [Q, Q], [150, 90], 16, 8, 128, 16, DT, 810, token_scale_range=(0.1, 10.0))
    small = GpuRun(wl).write_cache().attention()
    row = kvq().cache_row_bytes(DT, 128)
    nb = 4_600_000_000 // (16 * 8 * row)
    shift = nb - wl.num_blocks
    kc = torch.empty((nb, 16, 8, row), dtype=torch.uint8, device="cuda:0")
    vc = torch.empty_like(kc)
    assert kc.numel() > 2 ** 32
    far = GpuRun(wl)
    far.kc, far.vc = kc, vc
    far.slots += shift * 16
    far.bt[far.bt >= 0] += shift
    s, ws, write, attn = _prepared(far)
    write()
    attn()
    torch.cuda.synchronize()
    s.check_device()
    assert torch.equal(_bits(far.out), _bits(small.out))
    slots = wl.slot_mapping.to("cuda:0")
    assert torch.equal(kc.flatten(0, 1)[slots + shift * 16], small.kc.flatten(0, 1)[slots])
    k1, k2 = (torch.empty((slots.numel(), 8, 128), dtype=torch.float32, device="cuda:0") for _ in range(2))
    v1, v2 = torch.empty_like(k1), torch.empty_like(k1)
    kvq().gather_cache(kc, vc, far.slots, k1, v1, DT)
    kvq().gather_cache(small.kc, small.vc, slots, k2, v2, DT)
    assert torch.equal(k1, k2) and torch.equal(v1, v2)


def test_requests_without_new_tokens_and_padded_rows(cuda_device):
    """A request with no query, and rows of q and out behind the last
    sequence: left as they were."""
    wl = W.custom("int4-pad", [1, 0, 2], [40, 25, 300], 8, 2, 128, 16, DT, 820)
    g = GpuRun(wl).write_cache()
    g.attention()
    want = g.out.clone()
    pad = 5
    q = torch.full((wl.q.shape[0] + pad,) + tuple(wl.q.shape[1:]), float("nan"), dtype=torch.bfloat16,
                   device=g.dev)
    q[: wl.q.shape[0]] = g.q
    out = torch.full_like(q, 7.0)
    g.q, g.out = q, out
    s, ws, write, attn = _prepared(g)
    attn()
    torch.cuda.synchronize()
    assert torch.equal(_bits(out[: -pad]), _bits(want))
    assert torch.all(out[-pad:] == 7.0)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("mul", [2.0 ** 120, 2.0 ** 125, 2.0 ** -110])
def test_largest_and_smallest_values(cuda_device, D, mul):
    """Value rows at both ends of bf16's range (scales up to 2^118), whole and
    cut tiles, decode and prefill rows, among them a request of one key."""
    wl = W.custom("int4-range", [1, 30, 1, 1, 40], [1, 90, 77, 3000, 40], 8, 2, D, 16, DT, 830 + D)
    # (|x| < 6: the largest finite bf16 is 2^128 (1 - 2^-8))
    wl.value = (wl.value.float().clamp(-5.5, 5.5) * mul).to(torch.bfloat16)
    assert torch.isfinite(wl.value.float()).all()
    g = GpuRun(wl).write_cache()
    kc, vc = oracle_cache(wl)
    assert np.array_equal(g.vc.cpu().numpy(), vc)
    g.attention()
    ref, bnd = oracle_reference(wl, kc, vc)
    out = g.out_f32()
    assert np.isfinite(out).all()
    if mul > 1:
        assert_attention_close(out, ref, wl.name, bnd)
    else:
        # the bound of _harness.py, without its absolute floor of 1e-2
        tol = np.abs(ref) * 2.0 ** -8 + 2 * bnd + 2.0 ** -133
        assert (np.abs(out - ref) <= tol).all()


@pytest.mark.parametrize("D", [64, 128, 256])
def test_step_at_the_largest_values(cuda_device, D):
    wl = W.custom("int4-range-step", [1, 2, 1], [1, 90, 3000], 8, 2, D, 16, DT, 840 + D)
    wl.value = (wl.value.float().clamp(-5.5, 5.5) * 2.0 ** 125).to(torch.bfloat16)
    Step(wl).run().check(wl.name)


def test_caches_at_16_byte_offsets(cuda_device):
    wl = _mixed(850)
    want = GpuRun(wl).write_cache().attention()
    g = GpuRun(wl)
    n = g.kc.numel()
    for name in ("kc", "vc"):
        buf = torch.empty(n + 64, dtype=torch.uint8, device=g.dev)
        setattr(g, name, buf[16:16 + n].view(want.kc.shape))
        assert getattr(g, name).data_ptr() % 32 == 16
    s, ws, write, attn = _prepared(g)
    write()
    attn()
    torch.cuda.synchronize()
    s.check_device()
    assert torch.equal(_bits(g.out), _bits(want.out))
    slots = g.slots
    assert torch.equal(g.vc.flatten(0, 1)[slots], want.vc.flatten(0, 1)[slots])


def test_static_scratch(cuda_device):
    wl = _mixed(860)
    want = GpuRun(wl).write_cache().attention()
    k = kvq()
    s = k.get_scheduler_metadata(wl.num_req, wl.heads_q, wl.heads_kv, wl.head_dim, wl.seq_lens_t.numpy(),
                                 wl.query_start_loc.numpy(), wl.causal, wl.window, DT)
    out = torch.full_like(want.out, float("nan"))
    k.attention_with_kv_cache_static_scratch(s, want.q, want.kc, want.vc, want.qsl, want.sl, want.bt, wl.sm_scale,
                                             wl.causal, wl.window, wl.soft_cap, 1.0, 1.0, out, DT, wl.heads_kv)
    torch.cuda.synchronize()
    s.check_device()
    assert torch.equal(_bits(out), _bits(want.out))


CHILD = r"""
import os, sys
import numpy as np, torch
sys.path.insert(0, os.environ["KVQ_TEST_DIR"])
sys.path.insert(0, os.path.dirname(os.environ["KVQ_TEST_DIR"]))
from int8_kv_cache_reshape_gb300 import kvq
from test_gpu_int4_serving import Step, GpuRun, _mixed, W, DT
assert kvq.LIB_PATH.endswith("libkvq_checked.so"), kvq.LIB_PATH
g = GpuRun(_mixed(870)).write_cache().attention()
Step(W.custom("int4-checked-step", [1, 2], [500, 70], 8, 2, 128, 16, DT, 871)).run().check("checked step")
np.save(os.environ["KVQ_OUT"], g.out.view(torch.int16).cpu().numpy())
"""


def test_bounds_checked_build(cuda_device, tmp_path):
    """The build with the kernels' index checks gives the same bits."""
    import os
    import subprocess
    import sys
    from int8_kv_cache_reshape_gb300 import build as kvq_build
    here = os.path.dirname(os.path.abspath(__file__))
    env = dict(os.environ, KVQ_LIBRARY=str(kvq_build.build(checked=True)), KVQ_TEST_DIR=here,
               KVQ_OUT=str(tmp_path / "o.npy"))
    subprocess.run([sys.executable, "-c", CHILD], env=env, check=True, timeout=600)
    want = GpuRun(_mixed(870)).write_cache().attention()
    assert np.array_equal(np.load(tmp_path / "o.npy"), want.out.view(torch.int16).cpu().numpy())


class _Rewrite(Step):
    """A step whose new rows include rows of the context: every 13th token's,
    and those of blocks that a second request shares."""

    def __init__(self, wl, every):
        super().__init__(wl)
        pick = wl.new_token_mask()
        pick[::every] = True
        idx = torch.nonzero(pick).flatten()
        dev = self.g.dev
        # garbage (NaN scales) where the step is to write
        slots = wl.slot_mapping[idx].to(dev)
        self.g.kc.flatten(0, 1)[slots] = 0xFF
        self.g.vc.flatten(0, 1)[slots] = 0xFF
        self.nkey = wl.key[idx].contiguous().to(dev)
        self.nval = wl.value[idx].contiguous().to(dev)
        self.nslot = wl.slot_mapping[idx].contiguous().to(dev)


@pytest.mark.parametrize("D,every", [(128, 101), (64, 13), (256, 997), (128, 40)])
def test_step_that_rewrites_its_context(cuda_device, D, every):
    """Rows written anywhere are seen (fewer and more of them than the kernel
    looks through)."""
    for seed in range(3):
        wl = W.custom("int4-rewrite", [1, 2, 1, 1], [3000, 700, 2048, 40], 32, 8, D, 16, DT, 880 + seed)
        for _ in range(2):
            _Rewrite(wl, every).run().check(f"{wl.name} {every}")


def test_step_over_shared_blocks(cuda_device):
    """A new row in a block that another request's table holds too."""
    wl = W.custom("int4-shared", [1, 1], [520, 520], 8, 2, 128, 16, DT, 890)
    st = Step(wl)
    # request 1 reads request 0's blocks: its own new row goes to the same slot
    st.g.bt[1] = st.g.bt[0]
    st.nkey[1], st.nval[1], st.nslot[1] = st.nkey[0], st.nval[0], st.nslot[0]
    st.g.q[1] = st.g.q[0]
    # (not bit for bit between the two: the step cuts the chunks of the two
    # requests at different places, so their partial sums join in another order;
    # each is within the bound of _harness.py of request 0's exact result)
    kc, vc = oracle_cache(wl)
    ref, bnd = oracle_reference(wl, kc, vc, tokens=[0])
    for _ in range(5):
        st.g.out.fill_(float("nan"))
        st.run()
        torch.cuda.synchronize()
        kvq().decode_step_check(st.ws.t)
        for r in (0, 1):
            assert_attention_close(st.g.out_f32([r]), ref, f"request {r}", bnd)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_captured_step_with_new_lengths(cuda_device, D):
    """One captured step replayed, call after call without a synchronisation,
    for two batches in turn: lengths, tables, slots, new rows and q copied
    into place on the stream."""
    lens = ([900, 40, 3200, 300, 1, 1500], [1700, 2, 600, 3100, 45, 900])
    nb = 700
    wls = [W.custom(f"int4-replay-{i}", [1] * 6, L, 16, 4, D, 16, DT, 900 + i, token_scale_range=(0.1, 10.0),
                    num_blocks=nb) for i, L in enumerate(lens)]
    width = max(w.block_table.shape[1] for w in wls)
    direct = [Step(w).run() for w in wls]
    for d, w in zip(direct, wls):
        d.check(w.name)
    st = Step(wls[0])
    g = st.g
    g.bt = torch.full((6, width), -1, dtype=torch.int32, device=g.dev)
    g.bt[:, : wls[0].block_table.shape[1]] = wls[0].block_table.to(g.dev)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        st.run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        st.run()
    src = []
    for w in wls:
        s = Step(w)  # (its caches hold the context without the new rows)
        bt = torch.full((6, width), -1, dtype=torch.int32, device=g.dev)
        bt[:, : w.block_table.shape[1]] = w.block_table.to(g.dev)
        src.append((s, bt))
    got = []
    torch.cuda.synchronize()
    for i in (1, 0, 1, 1, 0):
        s, bt = src[i]
        g.kc.copy_(s.g.kc), g.vc.copy_(s.g.vc), g.bt.copy_(bt)
        for n in ("q", "qsl", "sl"):
            getattr(g, n).copy_(getattr(s.g, n))
        for n in ("nkey", "nval", "nslot"):
            getattr(st, n).copy_(getattr(s, n))
        g.out.fill_(float("nan"))
        graph.replay()
        got.append((i, g.out.clone(), g.vc.clone()))
    torch.cuda.synchronize()
    kvq().decode_step_check(st.ws.t)
    for i, out, vc in got:
        assert torch.equal(_bits(out), _bits(direct[i].g.out))
        assert torch.equal(vc, direct[i].g.vc)


def test_two_schedules_share_a_workspace(cuda_device):
    """Calls of different batches in turn on one stream and workspace."""
    parts = []
    for i, (ql, sl) in enumerate((([1, 1, 2], [3000, 700, 90]), ([1] * 9, [400] * 9), ([60, 1], [200, 2000]))):
        w = W.custom(f"int4-share-{i}", ql, sl, 16, 4, 128, 16, DT, 920 + i, token_scale_range=(0.1, 10.0))
        want = GpuRun(w).write_cache().attention().out.clone()
        g = GpuRun(w).write_cache()
        k = kvq()
        s = k.get_scheduler_metadata(w.num_req, 16, 4, 128, w.seq_lens_t.numpy(), w.query_start_loc.numpy(), True,
                                     w.window, DT)
        parts.append((g, s, want))
    ws = torch.zeros(max(s.workspace_bytes for _, s, _ in parts), dtype=torch.uint8, device="cuda:0")
    for _ in range(20):
        for g, s, _ in parts:
            w = g.wl
            g.out.fill_(float("nan"))
            kvq().attention_with_kv_cache(s, g.q, g.kc, g.vc, g.qsl, g.sl, g.bt, w.sm_scale, True, w.window,
                                          w.soft_cap, 1.0, 1.0, g.out, ws, DT, 4)
    torch.cuda.synchronize()
    for g, s, want in parts:
        s.check_device()
        assert torch.equal(_bits(g.out), _bits(want))
