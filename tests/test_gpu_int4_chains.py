"""Chains of 4-bit calls on one stream without a synchronisation between
them: the caches, the rows read back and the outputs of every step against
the same step run alone, bit for bit."""
import pytest
import torch

from _harness import GpuRun, kvq
from test_gpu_int4_serving import DT, _bits, _mixed, _prepared

pytestmark = pytest.mark.gpu

INPUTS = ("q", "key", "value", "slots", "bt")


def _alone(wl, dtype):
    """Output and the written slots' rows of K and V, as bytes and as values."""
    g = GpuRun(wl).write_cache().attention()
    rows = [torch.empty(tuple(wl.key.shape), dtype=dtype, device=g.dev) for _ in range(2)]
    kvq().gather_cache(g.kc, g.vc, g.slots, rows[0], rows[1], DT)
    torch.cuda.synchronize()
    return (g.out.clone(), g.kc.flatten(0, 1)[g.slots], g.vc.flatten(0, 1)[g.slots], *rows)


def _inputs(wl, dev):
    return dict(zip(INPUTS, (t.to(dev) for t in (wl.q, wl.key, wl.value, wl.slot_mapping, wl.block_table))))


def _check(got, want):
    out, k, v, rows, rows_v = got
    assert torch.equal(_bits(out), _bits(want[0]))
    assert torch.equal(k, want[1]) and torch.equal(v, want[2])
    assert torch.equal(rows, want[3]) and torch.equal(rows_v, want[4])


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_every_step_of_a_chain(cuda_device, D, dtype):
    runs = [_mixed(1100 + i, D) for i in range(6)]
    want = [_alone(w, dtype) for w in runs]
    g = GpuRun(runs[0])
    s, ws, write, attn = _prepared(g)
    src = [_inputs(w, g.dev) for w in runs]
    rows, rows_v = (torch.empty(tuple(runs[0].key.shape), dtype=dtype, device=g.dev) for _ in range(2))
    read = kvq().prepare_gather_cache(g.kc, g.vc, g.slots, rows, rows_v, DT)
    torch.cuda.synchronize()
    got = []
    for _ in range(3):
        for x in src:
            # (stale data of the step before would be seen)
            for t in (g.out, rows, rows_v):
                t.fill_(float("nan"))
            g.kc.fill_(0xFF), g.vc.fill_(0xFF)
            for n in INPUTS:
                getattr(g, n).copy_(x[n])
            write()
            attn()
            read()
            got.append((g.out.clone(), g.kc.flatten(0, 1)[g.slots], g.vc.flatten(0, 1)[g.slots], rows.clone(),
                        rows_v.clone()))
    torch.cuda.synchronize()
    s.check_device()
    for i, x in enumerate(got):
        _check(x, want[i % len(runs)])


def test_every_replay_of_a_captured_chain(cuda_device):
    k = kvq()
    runs = [_mixed(1120), _mixed(1121), _mixed(1122)]
    want = [_alone(w, torch.bfloat16) for w in runs]
    g = GpuRun(runs[0])
    rows, rows_v = (torch.empty(tuple(runs[0].key.shape), dtype=torch.bfloat16, device=g.dev) for _ in range(2))
    side = torch.cuda.Stream()
    s, ws, write, attn = _prepared(g, stream=side.cuda_stream)
    with torch.cuda.stream(side):
        write(), attn()                           # (the plan's upload stays out of the graph)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            write()
            attn()
            k.gather_cache(g.kc, g.vc, g.slots, rows, rows_v, DT, stream=side.cuda_stream)
    src = [_inputs(w, g.dev) for w in runs]
    got = []
    torch.cuda.synchronize()
    for i in (1, 0, 2, 2, 1, 0):
        for t in (g.out, rows, rows_v):
            t.fill_(float("nan"))
        g.kc.fill_(0xFF), g.vc.fill_(0xFF)
        for n in INPUTS:
            getattr(g, n).copy_(src[i][n])
        graph.replay()
        got.append((i, (g.out.clone(), g.kc.flatten(0, 1)[g.slots], g.vc.flatten(0, 1)[g.slots], rows.clone(),
                        rows_v.clone())))
    torch.cuda.synchronize()
    s.check_device()
    for i, x in got:
        _check(x, want[i])
