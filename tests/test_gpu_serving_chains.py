"""The calls of a serving loop together, one stream, no synchronisation
between them: tables, rotated rows into the cache, attention behind a shared
prefix or to an encoder.  The cache's bytes against the definition, the outputs
against the oracle over them."""
import numpy as np
import pytest
import torch

import _rotary as R
import oracle
from _harness import FILL, ORACLE_DT, Guarded, assert_attention_close, kvq
from _shared import CrossRun, SharedRun, compare, shared_workload
from int8_kv_cache_reshape_gb300 import workloads as W

pytestmark = pytest.mark.gpu

BLOCK, SCALES = 16, (0.013, 0.021)


class Server:
    """A pool, its free list and the device buffers of steps of up to `most` tokens."""

    def __init__(self, dtype, Hq, Hkv, D, device, requests, most=64, blocks=96, interleaved=False):
        self.dtype, self.shape, self.dev, self.n = dtype, (Hq, Hkv, D), device, requests
        row = kvq().cache_row_bytes(dtype, D)
        self.kc, self.vc = (Guarded((blocks, BLOCK, Hkv, row), torch.uint8, FILL, device) for _ in range(2))
        self.scales = SCALES if dtype in ("fp8_e4m3", "fp8_e5m2") else (1.0, 1.0)
        i32 = lambda *n: torch.zeros(n, dtype=torch.int32, device=device)  # noqa: E731
        self.free = torch.randperm(blocks, generator=torch.Generator().manual_seed(3)).to(device, torch.int32)
        self.free_count, self.status, self.bt = i32(1) + blocks, i32(4), i32(requests, 40) - 1
        self.qsl, self.sl = i32(requests + 1), i32(requests)
        self.slots, self.pos = (torch.zeros(most, dtype=torch.int64, device=device) for _ in range(2))
        self.qkv = torch.zeros((most, Hq + 2 * Hkv, D), dtype=torch.bfloat16, device=device)
        self.out = Guarded((most, Hq, D), torch.bfloat16, float("nan"), device)
        self.table = R.cos_sin_table(1000, D)
        self.cos_sin = torch.from_numpy(self.table).to(device)
        self.interleaved, self.lens = interleaved, [0] * requests
        self.gen = torch.Generator().manual_seed(5)
        self.queries, self.want = None, {}

    def load(self, new):
        """The next `new[r]` tokens of each request: lengths, positions and projections."""
        T, Hq = sum(new), self.shape[0]
        pos = np.concatenate([np.arange(n) + at for n, at in zip(new, self.lens)])
        self.lens = [a + n for a, n in zip(self.lens, new)]
        self.new, self.T = new, T
        qsl = np.concatenate([[0], np.cumsum(new)])
        self.qsl.copy_(torch.from_numpy(qsl.astype(np.int32)))
        self.sl.copy_(torch.tensor(self.lens, dtype=torch.int32))
        self.pos.fill_(-1)          # (the padded tail's)
        self.pos[:T] = torch.from_numpy(pos).to(self.dev)
        x = torch.randn(self.qkv.shape, generator=self.gen).to(torch.bfloat16)
        self.qkv.copy_(x)
        self.out.t.fill_(float("nan"))
        d = x[:T].double().numpy()
        Hkv = self.shape[1]
        turned = R.rotate(d[:, :Hq + Hkv], self.table, pos, self.interleaved)
        self.rows = (R.rows(self.dtype, turned[:, Hq:], self.scales[0]), R.rows(self.dtype, d[:, Hq + Hkv:], self.scales[1]))
        self.turned_q = R.bf16_bits(turned[:, :Hq])

    def tables(self):
        kvq().build_block_tables(self.qsl, self.sl, self.free, self.free_count, self.bt, self.slots, BLOCK,
                                 self.kc.t.shape[0], self.free_count, self.status)

    def append(self):
        Hq, Hkv, _ = self.shape
        q = self.qkv[:, :Hq]        # (rotated where it lies)
        kvq().rotary_and_cache(q, self.qkv[:, Hq:Hq + Hkv], self.qkv[:, Hq + Hkv:], self.pos, self.cos_sin, q, self.kc.t,
                               self.vc.t, self.slots, self.dtype, self.interleaved, *self.scales)

    def queries_side_by_side(self):
        return self.qkv[:, :self.shape[0]].contiguous()

    def attend(self, sched, ws, q):
        kvq().attention_with_kv_cache(sched, q, self.kc.t, self.vc.t, self.qsl, self.sl, self.bt, 0.1, True, 0, 0.0,
                                      *self.scales, self.out.t, ws, self.dtype, self.shape[1])

    def check(self, what):
        torch.cuda.synchronize()
        for g in (self.kc, self.vc, self.out):
            g.check(what)
        Hq, Hkv, _ = self.shape
        slots = self.slots.cpu().numpy()
        assert (slots[:self.T] >= 0).all() and (slots[self.T:] == -1).all() and self.status[:2].tolist() == [0, 0]
        for cache, rows in zip((self.kc, self.vc), self.rows):
            got = cache.t.cpu().numpy().reshape(-1, Hkv, rows.shape[-1])
            assert np.array_equal(got[slots[:self.T]], rows), what
        q = self.qkv[:, :Hq].cpu().view(torch.int16).numpy()
        assert np.array_equal(q[:self.T], self.turned_q) and not q[self.T:].any(), what
        out = self.out.t.float().cpu().numpy()
        assert np.isnan(out[self.T:]).all(), f"{what}: rows behind the last token"
        args = (self.turned_q.view(np.uint16), self.kc.t.cpu().numpy(), self.vc.t.cpu().numpy(), self.qsl.cpu(),
                self.sl.cpu(), self.bt.cpu().numpy(), Hkv, BLOCK, ORACLE_DT[self.dtype], 0.1, True, 0, 0.0, *self.scales)
        assert_attention_close(out[:self.T], oracle.attention(*args), what, oracle.attention_fp32_bound(*args))


@pytest.mark.parametrize("dtype,Hq,Hkv,D", [
    ("auto", 8, 2, 128), ("fp8_e4m3", 6, 6, 64), ("fp8_e5m2_per_token_head", 8, 1, 256),
    ("int8_per_token_head", 8, 2, 128), ("int4_per_token_head", 10, 2, 64)])
def test_samples_of_one_prompt(cuda_device, monkeypatch, dtype, Hq, Hkv, D):
    """A prompt is appended and attended to, then continued by six requests that
    hold its whole blocks together and a last block each; three of the steps have
    a padded tail, and the second last appends two tokens to some."""
    monkeypatch.setenv("KVQ_PREFIX_MIN_BYTES", "0")
    k, n, P = kvq(), 6, 141
    s = Server(dtype, Hq, Hkv, D, cuda_device, n, most=P + 5, interleaved=dtype == "fp8_e4m3")
    none = [0] * (n - 1)

    def step(new, sched, what):
        ws = torch.full((max(256, sched.workspace_bytes),), 0xFF, dtype=torch.uint8, device=cuda_device)
        s.tables()
        s.append()
        s.attend(sched, ws, s.queries_side_by_side())
        s.check(what)
        sched.check_device()
        sched.close()

    s.load([P] + none)
    step([P] + none, k.get_scheduler_metadata(n, Hq, Hkv, D, s.lens, s.qsl.cpu().numpy(), True, 0, dtype), "prompt")
    # the others begin with it: its whole blocks, and a copy of the last one
    whole = P // BLOCK
    last = s.bt[0, whole].clone()
    for r in range(1, n):
        s.bt[r, :whole] = s.bt[0, :whole]
        s.free_count -= 1
        new = s.free[s.free_count.long()]
        s.bt[r, whole] = new
        for c in (s.kc.t, s.vc.t):
            c[new.long()] = c[last.long()].clone()
        s.lens[r] = P
    for i, new in enumerate([[1] * n, [1] * n, [2, 1, 1, 2, 1, 0], [1, 1, 0, 1, 1, 1]]):
        s.load(new)
        sched = k.get_shared_prefix_metadata(n, Hq, Hkv, D, s.lens, s.qsl.cpu().numpy(), [P], [0] * n, 0, dtype)
        assert sched.rect_info()["num_shared_requests"] >= n - 1 and sched.rect_info()["num_units"] > 0
        step(new, sched, f"step {i}")


def test_a_captured_step_and_the_step_of_the_device_lengths(cuda_device, monkeypatch):
    """tables, rows and attention as one graph, replayed on other projections;
    then the same rows through decode_step without new rows of its own, which
    reads the lengths on the device."""
    monkeypatch.setenv("KVQ_PREFIX_MIN_BYTES", "0")
    k, n, dtype, Hq, Hkv, D = kvq(), 5, "int8_per_token_head", 8, 2, 128
    s = Server(dtype, Hq, Hkv, D, cuda_device, n, most=160)
    s.load([150, 0, 0, 0, 0])
    s.tables(), s.append()
    torch.cuda.synchronize()
    for r in range(1, n):
        s.bt[r] = s.bt[0]
        s.lens[r] = 144
    s.lens[0] = 144
    s.bt[:, 9:] = -1
    s.load([1, 2, 1, 1, 2])
    lens, state = list(s.lens), (s.free_count.clone(), s.bt.clone())
    sched = k.get_shared_prefix_metadata(n, Hq, Hkv, D, s.lens, s.qsl.cpu().numpy(), [144], [0] * n, 0, dtype)
    ws = torch.full((sched.workspace_bytes,), 0xFF, dtype=torch.uint8, device=cuda_device)
    q = torch.empty((160, Hq, D), dtype=torch.bfloat16, device=cuda_device)

    def step():
        s.tables()
        s.append()
        q.copy_(s.qkv[:, :Hq])
        s.attend(sched, ws, q)

    def again():
        s.free_count.copy_(state[0]), s.bt.copy_(state[1])

    step()
    s.check("first")
    graph = torch.cuda.CUDAGraph()
    again()
    with torch.cuda.graph(graph):
        step()
    for i in range(3):
        s.lens = [a - b for a, b in zip(lens, s.new)]
        again()
        s.load(s.new)
        graph.replay()
        s.check(f"replay {i}")
    sched.check_device()
    sched.close()
    # (no rows to store: they are in the cache)
    empty = torch.empty((0, Hkv, D), dtype=torch.bfloat16, device=cuda_device)
    zero = torch.zeros(k.decode_step_workspace_size(n, Hq, Hkv, D, dtype, 2), dtype=torch.uint8, device=cuda_device)
    s.out.t.fill_(float("nan"))
    k.decode_step(empty, empty, torch.empty(0, dtype=torch.int64, device=cuda_device), s.kc.t, s.vc.t, q, s.qsl, s.sl, s.bt,
                  2, 0.1, 0, 0.0, 1.0, 1.0, s.out.t, zero, dtype, Hkv)
    s.check("decode_step")
    k.decode_step_check(zero)


@pytest.mark.parametrize("dtype", ["auto", "int4_per_token_head"])
def test_a_decoder_with_both_attentions(cuda_device, dtype):
    """Causal attention to the decoder's own cache, then cross attention of
    the same tokens, two schedules on one workspace, captured together."""
    k, new, lens = kvq(), [3, 70, 1, 20], [200, 33, 0, 77]
    own = W.custom("own", new, [n + 40 for n in new], 8, 2, 128, 16, dtype, 9)
    enc = W.custom("enc", new, lens, 8, 2, 128, 16, dtype, 10, causal=False)
    a, b = SharedRun(own).write_cache(), CrossRun(enc).write_cache()
    own.prefix_lens, own.of = [], [-1] * 4
    sa, sb = a.schedule(), b.schedule()
    ws = torch.full((max(sa.workspace_bytes, sb.workspace_bytes),), 0xFF, dtype=torch.uint8, device=cuda_device)

    def call():
        for g, sched, causal in ((a, sa, True), (b, sb, False)):
            w = g.wl
            k.attention_with_kv_cache(sched, g.q, g.kc, g.vc, g.qsl, g.sl, g.bt, w.sm_scale, causal, 0, 0.0, 1.0, 1.0,
                                      g.out, ws, dtype, 2)

    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for g in (a, b):
        g.out.fill_(float("nan"))
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    compare(a, "own")
    compare(b, "cross")
    for s in (sa, sb):
        s.check_device()
        s.close()


@pytest.mark.parametrize("dtype,D", [("auto", 128), ("int8_per_token_head", 256), ("int4_per_token_head", 128)])
@pytest.mark.parametrize("cross", [False, True])
def test_pools_beyond_4_gib(cuda_device, monkeypatch, dtype, D, cross):
    """The blocks at the end of a pool of more than 2^32 bytes."""
    monkeypatch.setenv("KVQ_PREFIX_MIN_BYTES", "0")
    if cross:
        g = CrossRun(W.custom("far", [1, 60, 5], [90, 200, 300], 16, 8, D, 16, dtype, 4, causal=False))
    else:
        g = SharedRun(shared_workload([160], [0] * 4, [9, 1, 40, 20], [1] * 4, 16, 8, D, 16, dtype, 4))
    g.write_cache().attention()
    want = g.out.clone()
    near = g.kc.shape[0]
    blocks = (1 << 32) // g.kc[0].numel() + 3 + near
    far = []
    for c in (g.kc, g.vc):
        t = torch.zeros((blocks, *c.shape[1:]), dtype=torch.uint8, device=cuda_device)
        t[blocks - near:] = c
        far.append(t)
    g.kc, g.vc = far
    g.bt += blocks - near
    g.out.fill_(float("nan"))
    g.attention()
    assert torch.equal(g.out, want)


def test_tokens_beyond_4_gib(cuda_device):
    """Rows of queries beyond 2^31 elements: one vector a head, but the last
    129, which are a small batch's."""
    k, Hq, D, T, L = kvq(), 32, 256, (1 << 31) // (32 * 256) + 133, 70
    wl = W.custom("many", [64, 1, 64], [L, L, L], Hq, 4, D, 16, "fp8_per_token_head", 2, causal=False)
    small = CrossRun(wl).write_cache().attention()
    compare(small, "few tokens")
    big = torch.zeros((T, Hq, D), dtype=torch.bfloat16, device=cuda_device)
    out = torch.full_like(big, float("nan"))
    big[-129:] = small.q
    qsl = torch.tensor([0, T - 65, T - 64, T], dtype=torch.int32)
    big[:T - 129] = small.q[0]
    sched = k.get_cross_attention_metadata(3, Hq, 4, D, [L] * 3, qsl.numpy(), "fp8_per_token_head")
    ws = torch.full((max(256, sched.workspace_bytes),), 0xFF, dtype=torch.uint8, device=cuda_device)
    k.attention_with_kv_cache(sched, big, small.kc, small.vc, qsl.to(cuda_device), small.sl, small.bt, wl.sm_scale, False, 0,
                              0.0, 1.0, 1.0, out, ws, "fp8_per_token_head", 4)
    torch.cuda.synchronize()
    sched.check_device()
    sched.close()
    assert torch.equal(out[:T - 129].view(torch.int16), out[:1].view(torch.int16).expand(T - 129, -1, -1))
    for rows in (out[-129:], out[:129]):
        small.out.copy_(rows)
        compare(small, "rows of the large batch", tokens=range(129) if rows.data_ptr() != out.data_ptr() else [0])
