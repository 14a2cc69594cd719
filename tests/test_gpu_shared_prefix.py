"""Attention of batches that share prefixes, against the oracle (which reads
every request's context for itself)."""
import numpy as np
import pytest
import torch

from _harness import Guarded, GpuRun, kvq
from _shared import SharedRun, compare, shared_workload
from int8_kv_cache_reshape_gb300 import workloads as W

pytestmark = pytest.mark.gpu

DTYPES = ["auto", "fp8_e4m3", "fp8_e5m2", "int8_per_token_head", "fp8_per_token_head",
          "fp8_e5m2_per_token_head", "int4_per_token_head"]


@pytest.fixture(autouse=True)
def share_everything(monkeypatch):
    """4-bit batches as small as these would not be shared."""
    monkeypatch.setenv("KVQ_PREFIX_MIN_BYTES", "0")


def _run(wl, **kw):
    return SharedRun(wl, **kw).write_cache().attention()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("D,Hq,Hkv", [(64, 8, 2), (128, 8, 2), (256, 4, 1)])
def test_one_prefix(cuda_device, dtype, D, Hq, Hkv):
    own = [1, 2, 17, 40, 130, 5, 64, 300, 1]
    wl = shared_workload([400], [0] * 9, own, [1] * 9, Hq, Hkv, D, 16, dtype, 40 + D)
    g = _run(wl)
    assert g.rect["num_units"] > 0 and g.rect["num_shared_requests"] == 9 and g.rect["shared_keys"] == 9 * 384
    compare(g, f"{dtype} {D}")


@pytest.mark.parametrize("rows", ["one tile, part", "one tile, whole", "two tiles", "three tiles", "five tiles"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_row_tiles(cuda_device, rows, D):
    """Rows around the tiles' edges: 128 a row tile, 256 a unit."""
    R = {"one tile, part": 3, "one tile, whole": 32, "two tiles": 33, "three tiles": 65, "five tiles": 150}[rows]
    wl = shared_workload([160], [0] * R, [1 + (7 * r) % 23 for r in range(R)], [1] * R, 4, 1, D, 32,
                         "int8_per_token_head", R)
    g = _run(wl)
    assert g.rect["num_shared_requests"] == R
    compare(g, f"{rows} {D}")


@pytest.mark.parametrize("tiles", [1, 2, 3])
@pytest.mark.parametrize("P", [32, 96, 128, 129, 255, 1000, 1536])
@pytest.mark.parametrize("dtype,D", [("fp8_e4m3", 128), ("int4_per_token_head", 256), ("auto", 64)])
def test_cuts_of_the_prefix(cuda_device, monkeypatch, tiles, P, dtype, D):
    """KV tiles a unit, prefix lengths at and around tiles, chunks and blocks."""
    monkeypatch.setenv("KVQ_RECT_TILES", str(tiles))
    wl = shared_workload([P], [0] * 6, [3, 1, 50, 20, 9, 33], [1] * 6, 6, 2, D, 48, dtype, P + tiles)
    g = _run(wl)
    assert g.rect["num_units"] > 0
    compare(g, f"{P} keys, {tiles} tiles a unit")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("window,cap,alibi,sinks", [(0, 30.0, False, False), (300, 0.0, False, False),
                                                    (0, 0.0, True, True), (200, 50.0, True, True), (90, 0.0, False, True)])
def test_options(cuda_device, dtype, window, cap, alibi, sinks):
    """Windows that begin inside the prefix for some requests, inside its
    last tile for others, and after it for the rest."""
    own = [1, 33, 64, 100, 250, 299, 5, 180]
    wl = shared_workload([350], [0] * 8, own, [1] * 8, 8, 2, 128, 16, dtype, 3, window=window, soft_cap=cap)
    g = _run(wl, alibi_slopes=W.alibi_slopes(8) if alibi else None, sinks=W.sink_logits(8, 5) if sinks else None)
    compare(g, f"{dtype} window {window} cap {cap}")


@pytest.mark.parametrize("dtype", ["int8_per_token_head", "int4_per_token_head", "auto"])
def test_several_prefixes_and_kinds_of_requests(cuda_device, dtype):
    """Three prefixes (one of a single request, one of no keys), requests
    without one, verify steps of several tokens, a prompt that begins with a
    prefix, a request without new tokens; groups of five heads."""
    of = [0, 1, -1, 0, 1, 0, 2, -1, 0, 1, 3, 0]
    own = [4, 9, 120, 60, 3, 200, 11, 7, 90, 33, 20, 8]
    new = [1, 3, 1, 2, 3, 1, 1, 2, 70, 1, 1, 0]
    wl = shared_workload([260, 97, 64, 0], of, own, new, 10, 2, 128, 16, dtype, 9)
    g = _run(wl)
    assert g.rect["num_shared_requests"] == 6 and g.sched_info["num_prefill_tiles"] > 0
    compare(g, dtype)


def test_same_result_as_without_sharing(cuda_device):
    """Both plans of one batch agree to the rounding of their sums."""
    wl = shared_workload([512], [0] * 20, [1 + 3 * r for r in range(20)], [1] * 20, 8, 2, 128, 16, "fp8_e4m3", 77)
    a, b = _run(wl).out_f32(), GpuRun(wl).write_cache().attention().out_f32()
    # both are within half a bf16 step (2^-9 of the value) plus their fp32 sums of the exact result
    assert np.abs(a - b).max() <= 2.0 ** -7 * np.abs(b).max()


def test_small_batches_are_planned_without_sharing(cuda_device, monkeypatch):
    monkeypatch.delenv("KVQ_PREFIX_MIN_BYTES")
    for dtype, shared in (("int4_per_token_head", 0), ("int8_per_token_head", 4)):
        wl = shared_workload([256], [0] * 4, [3, 4, 5, 6], [1] * 4, 8, 2, 128, 16, dtype, 2)
        g = _run(wl)
        assert g.rect["num_shared_requests"] == shared and (g.rect["num_units"] > 0) == (shared > 0)
        compare(g, dtype)


def test_blocks_that_are_missing_from_the_table(cuda_device):
    """Entries outside the pool inside the prefix and inside a request's own keys."""
    wl = shared_workload([320], [0] * 5, [20, 40, 3, 60, 9], [1] * 5, 8, 2, 128, 16, "fp8_per_token_head", 4)
    g = SharedRun(wl).write_cache()
    wl.block_table[:, 3] = -1
    wl.block_table[:, 19] = wl.num_blocks + 5
    wl.block_table[1, 21] = -7
    g.bt.copy_(wl.block_table)
    g.attention()
    kc, vc = g.kc.cpu().numpy(), g.vc.cpu().numpy()
    x = wl
    keys = [[j for j in range(x.seq_lens[r]) if 0 <= x.block_table[r, j // 16] < x.num_blocks] for r in range(5)]
    got = g.out_f32()
    import oracle
    from _harness import ORACLE_DT
    dt = ORACLE_DT["fp8_per_token_head"]
    # gather the present rows into a pool of one block a request and attend there
    row = kc.shape[-1]
    width = -(-max(len(k) for k in keys) // 16)
    pk = np.zeros((5 * width, 16, 2, row), np.uint8)
    pv = np.zeros_like(pk)
    flat = lambda c: c.reshape(-1, 2, row)  # noqa: E731
    for r, ks in enumerate(keys):
        slots = [int(x.block_table[r, j // 16]) * 16 + j % 16 for j in ks]
        flat(pk)[r * width * 16: r * width * 16 + len(ks)] = flat(kc)[slots]
        flat(pv)[r * width * 16: r * width * 16 + len(ks)] = flat(vc)[slots]
    bt = np.arange(5 * width, dtype=np.int32).reshape(5, width)
    args = (W.bf16_bits(x.q), pk, pv, x.query_start_loc, torch.tensor([len(k) for k in keys], dtype=torch.int32),
            torch.from_numpy(bt), 2, 16, dt, x.sm_scale, False, 0, 0.0, 1.0, 1.0)
    from _harness import assert_attention_close
    assert_attention_close(got, oracle.attention(*args), "missing blocks", oracle.attention_fp32_bound(*args))


def test_what_lies_behind_the_keys_is_not_read(cuda_device):
    """Rows of the last blocks after the last key, and blocks of no request,
    hold NaN."""
    wl = shared_workload([200], [0] * 4, [5, 20, 1, 9], [1] * 4, 8, 2, 64, 64, "auto", 8)
    g = SharedRun(wl)
    for c in (g.kc, g.vc):
        c.fill_(0xFF)
    g.write_cache().attention()
    kc, vc = (np.zeros(tuple(c.shape), np.uint8) for c in (g.kc, g.vc))
    assert np.isfinite(g.out_f32()).all()
    compare(g, "NaN behind the keys")


@pytest.mark.parametrize("sm_scale", [0.0, -0.05])
@pytest.mark.parametrize("dtype", ["auto", "int8_per_token_head", "int4_per_token_head"])
def test_score_scales_of_zero_and_below(cuda_device, sm_scale, dtype):
    wl = shared_workload([300], [0] * 5, [5, 20, 1, 9, 40], [1] * 5, 8, 2, 128, 16, dtype, 8, sm_scale=sm_scale)
    compare(_run(wl), f"{dtype} {sm_scale}")


@pytest.mark.parametrize("dtype", ["int8_per_token_head", "fp8_per_token_head", "int4_per_token_head"])
@pytest.mark.parametrize("exponent", [-80, 90])
def test_value_scales_at_both_ends(cuda_device, dtype, exponent):
    """Values of 2^-80 and 2^90 (the 8-bit decode, which reads the requests' own
    keys, holds its reference within 2^-100 and 2^100)."""
    wl = shared_workload([260], [0] * 4, [5, 20, 1, 9], [1] * 4, 8, 2, 128, 16, dtype, 12)
    small = wl.value.float()
    wl.value = (small * 2.0 ** exponent).to(torch.bfloat16)
    g = _run(wl)
    out = torch.from_numpy(g.out_f32().astype(np.float64) * 2.0 ** -exponent)
    wl.value = small.to(torch.bfloat16)
    h = _run(wl)
    # a power of two on every value moves the row scales by it exactly, and so the output
    assert torch.equal(out.float(), torch.from_numpy(h.out_f32()))
    compare(h, dtype)


def test_zero_values_and_zero_keys(cuda_device):
    wl = shared_workload([150], [0] * 3, [4, 9, 1], [1] * 3, 8, 2, 128, 16, "int8_per_token_head", 12)
    wl.value.zero_()
    assert not _run(wl).out_f32().any()
    wl = shared_workload([150], [0] * 3, [4, 9, 1], [1] * 3, 8, 2, 128, 16, "fp8_per_token_head", 12)
    wl.key.zero_()
    compare(_run(wl), "zero keys")


def test_two_batches_of_one_schedule_and_two_streams(cuda_device):
    """A schedule used for two layers one after another, and two schedules
    with workspaces of their own on two streams at once."""
    wl = [shared_workload([700], [0] * 12, [5 * r + 1 for r in range(12)], [1] * 12, 8, 2, 128, 16, dt, s)
          for dt, s in (("int8_per_token_head", 1), ("int4_per_token_head", 2), ("int8_per_token_head", 3))]
    a, b, c = (SharedRun(w).write_cache() for w in wl)
    sched = a.schedule()
    a.attention(sched)
    c.attention(sched)
    sched.close()
    compare(a, "first layer")
    compare(c, "second layer")
    for g in (a, b):
        g.out.fill_(float("nan"))
    k, runs = kvq(), []
    for g in (a, b):
        s, sched = torch.cuda.Stream(), g.schedule()
        ws = Guarded((sched.workspace_bytes,), torch.uint8, 0xFF, cuda_device)
        runs.append((g, s, sched, ws))
    torch.cuda.synchronize()
    for _ in range(3):
        for g, s, sched, ws in runs:
            w = g.wl
            k.attention_with_kv_cache(sched, g.q, g.kc, g.vc, g.qsl, g.sl, g.bt, w.sm_scale, True, 0, 0.0, w.k_scale,
                                      w.v_scale, g.out, ws.t, w.kv_cache_dtype, w.heads_kv, stream=s)
    torch.cuda.synchronize()
    for g, s, sched, ws in runs:
        sched.check_device()
        ws.check("workspace")
        compare(g, "two streams")
        sched.close()


def test_reruns_are_bit_identical_and_captured(cuda_device):
    wl = shared_workload([900], [0] * 30, [3 * r + 1 for r in range(30)], [1] * 30, 8, 2, 128, 16,
                         "int8_per_token_head", 31)
    g = SharedRun(wl).write_cache()
    sched = g.schedule()
    ws = Guarded((sched.workspace_bytes,), torch.uint8, 0xFF, cuda_device)
    g.attention(sched, ws)
    first = g.out.clone()
    graph, k = torch.cuda.CUDAGraph(), kvq()
    with torch.cuda.graph(graph):
        k.attention_with_kv_cache(sched, g.q, g.kc, g.vc, g.qsl, g.sl, g.bt, wl.sm_scale, True, 0, 0.0, 1.0, 1.0, g.out,
                                  ws.t, wl.kv_cache_dtype, wl.heads_kv)
    for _ in range(3):
        g.out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(g.out, first)
    sched.check_device()
    sched.close()


def test_static_scratch(cuda_device):
    wl = shared_workload([500], [0] * 10, [7 * r + 1 for r in range(10)], [1] * 10, 8, 2, 128, 16, "fp8_e5m2", 6)
    g = SharedRun(wl).write_cache()
    sched = g.schedule()
    kvq().attention_with_kv_cache_static_scratch(
        sched, g.q, g.kc, g.vc, g.qsl, g.sl, g.bt, wl.sm_scale, True, 0, 0.0, wl.k_scale, wl.v_scale, g.out,
        wl.kv_cache_dtype, wl.heads_kv)
    torch.cuda.synchronize()
    sched.check_device()
    sched.close()
    compare(g, "static scratch")
