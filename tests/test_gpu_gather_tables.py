"""gather_cache (rows read back as values) and build_block_tables (block
tables and slot maps from device lengths) against plain restatements, and a
serving loop of all the 4-bit operators together.

gather: an fp32 output is code * scale, one rounding (the oracle's codes and
scales are bit-exact, so equality is required of fp32 products, and of their
bf16 roundings).  Tables are whole numbers: equality.
"""
import numpy as np
import pytest
import torch

import oracle
from int8_kv_cache_reshape_gb300 import workloads as W

from _harness import (FILL, GUARD_BYTES, Guarded, GpuRun, assert_attention_close, kvq, oracle_cache,
                      oracle_reference)

pytestmark = pytest.mark.gpu

DTYPES = ["auto", "fp8_e4m3", "fp8_e5m2", "int8_per_token_head", "fp8_per_token_head", "fp8_e5m2_per_token_head",
          "int4_per_token_head"]


def _values(rows, dtype, D, scale):
    """float32 values of cache rows (uint8 [..., row], numpy): codes decoded
    one by one, then one float32 product."""
    f = np.float32
    if dtype == "auto":
        return (np.ascontiguousarray(rows).view("<u2").astype(np.uint32) << 16).view(f)
    if dtype == "int4_per_token_head":
        w = np.ascontiguousarray(rows[..., : D // 2]).view("<u4")
        c = np.zeros(rows.shape[:-1] + (D,), f)
        for j in range(8):
            c[..., (2 * j if j < 4 else 2 * (j - 4) + 1)::8] = ((w >> (4 * j)) & 15).astype(f) - 8
        m = np.repeat(rows[..., D // 2 + 4: D // 2 + 12], D // 8, axis=-1).astype(f)
        s = np.ascontiguousarray(rows[..., D // 2: D // 2 + 4]).view("<f4")
        return s * (m * c)
    codes = rows[..., :D]
    if dtype == "int8_per_token_head":
        c = codes.view(np.int8).astype(f)
    else:
        fmt = oracle.E5M2 if "e5m2" in dtype else oracle.E4M3
        c = np.array([oracle.fp8_decode(fmt, i) for i in range(256)]).astype(f)[codes]
    s = np.ascontiguousarray(rows[..., D: D + 4]).view("<f4") if "per_token" in dtype else f(scale)
    return c * s


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("D,hkv", [(64, 3), (128, 8), (256, 1)])
@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
def test_gather_values(cuda_device, dtype, D, hkv, out):
    wl = W.custom("gather", [1, 1], [77, 20], hkv, hkv, D, 16, dtype, 500 + D, extra_blocks=2,
                  token_scale_range=(0.01, 100.0) if "per_token" in dtype else None)
    wl.key[3] = 0
    g = GpuRun(wl).write_cache()
    kc, vc = oracle_cache(wl)
    # out of order, twice the same, none, past the pool
    rng = np.random.default_rng(D)
    slots = np.concatenate([rng.permutation(wl.slot_mapping.numpy()), wl.slot_mapping.numpy()[[5, 5]],
                            [-1, wl.num_blocks * wl.block_size, -7]]).astype(np.int64)
    T = slots.size
    outs = [Guarded((T, hkv, D), out, float("nan"), g.dev) for _ in range(2)]
    kvq().gather_cache(g.kc, g.vc, torch.from_numpy(slots).to(g.dev), outs[0].t, outs[1].t, dtype, wl.k_scale,
                       wl.v_scale)
    torch.cuda.synchronize()
    live = (slots >= 0) & (slots < wl.num_blocks * wl.block_size)
    for o, cache, scale in ((outs[0], kc, wl.k_scale), (outs[1], vc, wl.v_scale)):
        o.check("gather output")
        flat = cache.reshape(-1, hkv, cache.shape[-1])
        want = _values(flat[np.where(live, slots, 0)], dtype, D, scale)
        want = torch.from_numpy(np.where(live[:, None, None], want, np.float32(0))).to(out)
        assert torch.equal(o.t.cpu(), want)


def test_gather_into_strided_rows(cuda_device):
    """Outputs as views of a wider buffer: the rest of it stays as it was."""
    wl = W.custom("gather-strided", [1], [50], 2, 2, 128, 16, "int4_per_token_head", 510)
    g = GpuRun(wl).write_cache()
    buf = torch.full((50, 7, 128), 3.0, device=g.dev)
    kvq().gather_cache(g.kc, g.vc, g.slots, buf[:, 1:3], buf[:, 4:6], "int4_per_token_head")
    a, b = torch.empty((50, 2, 128), device=g.dev), torch.empty((50, 2, 128), device=g.dev)
    kvq().prepare_gather_cache(g.kc, g.vc, g.slots, a, b, "int4_per_token_head")()
    assert torch.equal(buf[:, 1:3], a) and torch.equal(buf[:, 4:6], b)
    assert (buf[:, [0, 3, 6]] == 3.0).all()
    # outputs 16 bytes off a 32-byte border (16-byte stores)
    flat = torch.full((2 * 50 * 2 * 128 + 16,), 5.0, device=g.dev)
    c, d = (flat[4 + i * 12800: 4 + (i + 1) * 12800].view(50, 2, 128) for i in range(2))
    kvq().gather_cache(g.kc, g.vc, g.slots, c, d, "int4_per_token_head")
    assert torch.equal(c, a) and torch.equal(d, b)
    assert (flat[:4] == 5.0).all() and (flat[4 + 25600:] == 5.0).all()
    empty = torch.empty((0, 2, 128), device=g.dev)
    kvq().gather_cache(g.kc, g.vc, g.slots[:0], empty, empty, "int4_per_token_head")


# ---- block tables -----------------------------------------------------------------


def _plain_tables(ql, sl, free, count, table, slots_n, block, num_blocks):
    """The operator, one token at a time."""
    table = table.copy()
    slots = np.full(slots_n, -1, np.int64)
    count = max(0, min(count, len(free)))
    taken = bad = 0
    t = 0
    for r, (Q, L) in enumerate(zip(ql, sl)):
        need, held = -(-L // block), -(-(L - Q) // block)
        if Q > L or t + Q > slots_n or (Q > 0 and need > table.shape[1]):
            bad += 1
            t += Q
            continue
        if Q > 0:
            for lb in range(held, need):
                table[r, lb] = free[count - 1 - taken] if taken < count else -1
                taken += 1
        for i in range(Q):
            p = L - Q + i
            b = table[r, p // block]
            if 0 <= b < num_blocks:
                slots[t + i] = int(b) * block + p % block
        t += Q
    return table, slots, max(0, count - taken), max(0, taken - count), bad


def _tables_case(rng, ql, sl, block, spare=3, pad=0, width=None, drop=0):
    R = len(ql)
    need = [-(-L // block) for L in sl]
    width = max(1, max(need, default=1)) if width is None else width
    num_blocks = sum(need) + spare
    perm = rng.permutation(num_blocks).astype(np.int32)
    table = rng.integers(-5, num_blocks + 5, (max(1, R), width)).astype(np.int32)   # stale entries
    used = 0
    for r in range(R):
        held = min(width, -(-max(0, sl[r] - ql[r]) // block))
        table[r, :held] = perm[used: used + held]
        used += held
    free = perm[used:].copy()
    return dict(ql=ql, sl=sl, block=block, table=table, free=free, count=max(0, len(free) - drop),
                slots=sum(ql) + pad, num_blocks=num_blocks)


def _run_tables(c, dev, alias=False):
    R = len(c["ql"])
    i32 = lambda v: torch.tensor(np.asarray(v, np.int32), device=dev)  # noqa: E731
    table = Guarded(c["table"].shape, torch.int32, 0, dev)
    table.t.copy_(torch.from_numpy(c["table"]))
    slots = Guarded((c["slots"],), torch.int64, 123, dev)
    count = i32([c["count"]])
    left = count if alias else i32([-9])
    status = i32([0, 0, 0, 0])
    qsl = i32(np.concatenate([[0], np.cumsum(c["ql"])]))
    k = kvq()
    for _ in range(1 if alias else 2):      # (twice: a call leaves status ready for the next)
        k.build_block_tables(qsl, i32(c["sl"]), i32(c["free"]), count, table.t[:R] if R else table.t[:0], slots.t,
                             c["block"], c["num_blocks"], left, status)
    torch.cuda.synchronize()
    table.check("block table")
    slots.check("slot mapping")
    want = _plain_tables(c["ql"], c["sl"], c["free"], c["count"], c["table"], c["slots"], c["block"], c["num_blocks"])
    assert np.array_equal(table.t.cpu().numpy(), want[0])
    assert np.array_equal(slots.t.cpu().numpy(), want[1])
    assert int(left) == want[2]
    st = status.cpu().tolist()
    assert st[:3] == [want[3], want[4], 0]
    return want


@pytest.mark.parametrize("block", [1, 7, 16, 2176])
@pytest.mark.parametrize("R,max_q,max_l", [(1, 1, 1), (1, 1, 100), (64, 1, 4096), (5, 5000, 9000), (300, 3, 50),
                                           (700, 1, 3000), (3, 2000, 2000), (600, 40, 600)])
@pytest.mark.parametrize("alias", [False, True])
def test_tables(cuda_device, block, R, max_q, max_l, alias):
    rng = np.random.default_rng(R * 7 + max_q + block)
    sl = rng.integers(1, max_l + 1, R).tolist()
    if block == 1:
        sl = [min(x, 600) for x in sl]
    ql = [int(rng.integers(0, min(L, max_q) + 1)) for L in sl]
    if max_q == max_l:
        ql = list(sl)
    _run_tables(_tables_case(rng, ql, sl, block, pad=int(rng.integers(0, 2000))), cuda_device, alias)


def test_tables_edges(cuda_device):
    rng = np.random.default_rng(5)
    # no requests, no tokens
    _run_tables(_tables_case(rng, [], [], 16, pad=0), cuda_device)
    _run_tables(_tables_case(rng, [], [], 16, pad=3000), cuda_device)
    _run_tables(_tables_case(rng, [0, 0], [0, 40], 16), cuda_device)
    # lengths on the block border, first and last token of a block
    _run_tables(_tables_case(rng, [1, 1, 1, 16, 17, 1], [16, 17, 1, 16, 33, 32], 16), cuda_device)
    # runs of requests without tokens between others, at a CTA's border
    ql = [0] * 300 + [1024] + [0] * 300 + [1] * 500 + [0] * 5
    _run_tables(_tables_case(rng, ql, [q + int(rng.integers(0, 50)) for q in ql], 16), cuda_device)


@pytest.mark.parametrize("drop", [1, 7, 10 ** 6])
def test_tables_free_list_runs_out(cuda_device, drop):
    rng = np.random.default_rng(drop)
    sl = rng.integers(1, 200, 90).tolist()
    ql = [int(rng.integers(1, L + 1)) for L in sl]
    c = _tables_case(rng, ql, sl, 16, spare=0, drop=drop)
    _, slots, left, missing, bad = _run_tables(c, cuda_device)
    assert left == 0 and missing == min(drop, missing) > 0 and bad == 0 and (slots == -1).any()


def test_tables_requests_left_out(cuda_device):
    """More new tokens than keys, a table too narrow, tokens past the buffer:
    nothing is taken for them, the others go on."""
    rng = np.random.default_rng(6)
    ql, sl = [1, 5, 40, 3, 2], [30, 3, 400, 7, 90]
    c = _tables_case(rng, ql, sl, 16, spare=50, width=6)
    c["slots"] -= 1
    want = _run_tables(c, cuda_device)
    assert want[4] == 3
    # ids outside the pool give no slot
    c = _tables_case(rng, [4, 1], [20, 17], 16)
    c["free"][-1] = c["num_blocks"] + 1
    c["table"][1, 0] = -1
    _run_tables(c, cuda_device)


def test_tables_far_slots(cuda_device):
    """Slots beyond 32 bits: ids near 2^31 / 16 in blocks of 2176."""
    rng = np.random.default_rng(8)
    c = _tables_case(rng, [30, 1], [40, 2177], 2176)
    c["free"] = (c["free"] + 130_000_000).astype(np.int32)
    c["num_blocks"] = 131_000_000
    want = _run_tables(c, cuda_device)
    assert want[1].max() > 2 ** 37


def test_serving_loop(cuda_device):
    """Block tables, the fused step and rows read back, as a serving loop
    would run them, captured once and replayed with growing lengths; every
    step's output against the oracle over the cache so far."""
    k = kvq()
    dev, dt = cuda_device, "int4_per_token_head"
    hq, hkv, D, B, R, NB = 8, 2, 128, 16, 5, 40
    rng = np.random.default_rng(11)
    lens = np.array([0, 14, 15, 31, 60])
    g = torch.Generator().manual_seed(3)
    i32 = lambda v: torch.tensor(np.asarray(v, np.int32), device=dev)  # noqa: E731
    free, count, status = i32(rng.permutation(NB)), i32([NB]), i32([0] * 4)
    table = torch.full((R, 8), -1, dtype=torch.int32, device=dev)
    kc = torch.full((NB, B, hkv, D // 2 + 16), FILL, dtype=torch.uint8, device=dev)
    vc = kc.clone()
    # the prompts: tables, rows, and what was written read back
    qsl, sl = i32(np.concatenate([[0], np.cumsum(lens)])), i32(lens)
    T = int(lens.sum())
    keys = [torch.randn((T, hkv, D), generator=g).bfloat16(), torch.randn((T, hkv, D), generator=g).bfloat16()]
    slots = torch.zeros(T, dtype=torch.int64, device=dev)
    k.build_block_tables(qsl, sl, free, count, table, slots, B, NB, count, status)
    k.reshape_and_cache(keys[0].to(dev), keys[1].to(dev), kc, vc, slots, dt)
    back = [torch.empty((T, hkv, D), device=dev) for _ in range(2)]
    k.gather_cache(kc, vc, slots, back[0], back[1], dt)
    # a value is off by at most half a step of its group, at most amax / 14
    # (and the step's own rounding)
    for x, y in zip(keys, back):
        amax = x.float().abs().amax(-1, keepdim=True)
        assert ((y.cpu() - x.float()).abs() <= amax / 14 * (1 + 2.0 ** -6)).all()
    # single tokens: one captured step
    q, nk, nv = (torch.zeros((R, h, D), dtype=torch.bfloat16, device=dev) for h in (hq, hkv, hkv))
    out = torch.zeros_like(q)
    qsl1, slots1 = i32(range(R + 1)), torch.zeros(R + 2, dtype=torch.int64, device=dev)   # (padded by two)
    ws = torch.zeros(k.decode_step_workspace_size(R, hq, hkv, D, dt), dtype=torch.uint8, device=dev)
    nk2, nv2 = (torch.zeros((R + 2, hkv, D), dtype=torch.bfloat16, device=dev) for _ in range(2))

    def step(stream=None):
        k.build_block_tables(qsl1, sl, free, count, table, slots1, B, NB, count, status, stream=stream)
        k.decode_step(nk2, nv2, slots1, kc, vc, q, qsl1, sl, table, 1, D ** -0.5, 0, 0.0, 1.0, 1.0, out, ws, dt, hkv,
                      stream=stream)

    def fresh():
        for t in (q, nk2, nv2):
            t.copy_(torch.randn(t.shape, generator=g).bfloat16())

    def check():
        torch.cuda.synchronize()
        k.decode_step_check(ws)
        assert status.cpu().tolist()[:3] == [0, 0, 0]
        wl = W.custom("loop", [1] * R, lens.tolist(), hq, hkv, D, B, dt, 1)
        wl.q, wl.num_blocks = q.cpu(), NB
        wl.block_table = table.cpu()
        ref, bnd = oracle_reference(wl, kc.cpu().numpy(), vc.cpu().numpy())
        assert_attention_close(out.float().cpu().numpy(), ref, "serving loop", bnd)
        held = [table[r, : -(-int(L) // B)].cpu().tolist() for r, L in enumerate(lens)]
        ids = sum(held, [])
        assert len(set(ids)) == len(ids) and min(ids) >= 0            # no block twice
        assert int(count) == NB - len(ids)
        # the new rows are where the oracle writes them
        rk = np.full(kc.shape, FILL, np.uint8)
        rv = rk.copy()
        s = slots1.cpu().numpy()
        assert (s[R:] == -1).all()
        oracle.reshape_and_cache(W.bf16_bits(nk2), W.bf16_bits(nv2), rk, rv, s, oracle.INT4_PER_TOKEN_HEAD, 1.0, 1.0, B)
        for r in range(R):
            b, o = divmod(int(s[r]), B)
            assert np.array_equal(rk[b, o], kc[b, o].cpu().numpy()) and np.array_equal(rv[b, o], vc[b, o].cpu().numpy())

    stream = torch.cuda.Stream()
    lens += 1
    sl.copy_(i32(lens))
    fresh()
    with torch.cuda.stream(stream):
        stream.wait_stream(torch.cuda.default_stream())
        step(stream)
    check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        step(stream)
    for _ in range(4):
        lens += 1
        sl.copy_(i32(lens))
        fresh()
        torch.cuda.synchronize()
        graph.replay()
        check()
