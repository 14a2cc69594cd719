"""rotary_and_cache on the GPU: rotated queries and stored bytes, bit for bit
against the definition."""
import numpy as np
import pytest
import torch

import _rotary as R
from _harness import FILL, Guarded, kvq

pytestmark = pytest.mark.gpu

DTYPES = ["auto", "fp8_e4m3", "fp8_e5m2", "int8_per_token_head", "fp8_per_token_head",
          "fp8_e5m2_per_token_head", "int4_per_token_head"]


class Case:
    """A fused projection's output (rows at its stride), slots in random order."""

    def __init__(self, dtype, T, Hq, Hkv, D, rotary, interleaved, seed, block=16, max_position=5000, spread=1.0):
        g = torch.Generator().manual_seed(seed)
        rng = np.random.default_rng(seed)
        self.dtype, self.interleaved, self.shape = dtype, interleaved, (T, Hq, Hkv, D)
        qkv = torch.randn((T, Hq + 2 * Hkv, D), generator=g) * torch.exp(spread * torch.randn((T, 1, 1), generator=g))
        self.qkv = qkv.to(torch.bfloat16)
        self.table = R.cos_sin_table(max_position, rotary)
        self.positions = rng.integers(0, max_position, T)
        self.blocks = (T + block - 1) // block + 2
        self.block = block
        self.slots = rng.permutation(self.blocks * block)[:T]
        self.k_scale, self.v_scale = (0.013, 0.021) if dtype in ("fp8_e4m3", "fp8_e5m2") else (1.0, 1.0)

    def run(self, device, in_place=False, stream=None):
        T, Hq, Hkv, D = self.shape
        row = kvq().cache_row_bytes(self.dtype, D)
        self.kc = Guarded((self.blocks, self.block, Hkv, row), torch.uint8, FILL, device)
        self.vc = Guarded((self.blocks, self.block, Hkv, row), torch.uint8, FILL, device)
        qkv = self.qkv.to(device)
        q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        self.out = None if in_place else Guarded((T, Hq, D), torch.bfloat16, float("nan"), device)
        self.keep = (qkv, torch.from_numpy(np.asarray(self.positions, np.int64)).to(device),
                     torch.from_numpy(self.table).to(device),
                     torch.from_numpy(np.asarray(self.slots, np.int64)).to(device))
        kvq().rotary_and_cache(q, k, v, self.keep[1], self.keep[2], q if in_place else self.out.t, self.kc.t,
                               self.vc.t, self.keep[3], self.dtype, self.interleaved, self.k_scale, self.v_scale,
                               stream=stream)
        torch.cuda.synchronize()
        for t in (self.kc, self.vc, self.out):
            if t is not None:
                t.check("rotary_and_cache")
        # keys and values are inputs
        assert torch.equal(qkv[:, Hq:].cpu().view(torch.int16), self.qkv[:, Hq:].view(torch.int16))
        if not in_place:
            assert torch.equal(q.cpu().view(torch.int16), self.qkv[:, :Hq].view(torch.int16))
        return (q if in_place else self.out.t).cpu().view(torch.int16).numpy()

    def check(self, got):
        T, Hq, Hkv, D = self.shape
        x = self.qkv.double().numpy()
        pos = np.asarray(self.positions)
        known = (pos >= 0) & (pos < self.table.shape[0])
        turned = R.rotate(x[:, :Hq + Hkv], self.table, np.where(known, pos, 0), self.interleaved)
        want = np.where(known[:, None, None], R.bf16_bits(turned[:, :Hq]), 0)
        assert np.array_equal(got, want)
        slots = np.asarray(self.slots)
        live = known & (slots >= 0) & (slots < self.blocks * self.block)
        for cache, rows in ((self.kc, R.rows(self.dtype, turned[:, Hq:], self.k_scale)),
                            (self.vc, R.rows(self.dtype, x[:, Hq + Hkv:], self.v_scale))):
            want = np.full((self.blocks * self.block, Hkv, rows.shape[-1]), FILL, np.uint8)
            want[slots[live]] = rows[live]
            assert np.array_equal(cache.t.cpu().numpy().reshape(want.shape), want)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("D,rotary", [(64, 64), (64, 48), (128, 128), (128, 16), (256, 256), (256, 80)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_bytes_and_queries(cuda_device, dtype, D, rotary, interleaved):
    c = Case(dtype, 37, 6, 3 if D < 256 else 1, D, rotary, interleaved, 7 + D + rotary)
    # rows without a slot, past the pool, and positions outside the table
    c.slots[[0, 11]] = -1
    c.slots[20] = c.blocks * c.block
    c.positions[[5, 11]] = -1
    c.positions[6] = c.table.shape[0]
    c.positions[7] = 2 ** 40
    c.check(c.run(cuda_device, in_place=interleaved))


@pytest.mark.parametrize("T,Hq,Hkv", [(1, 1, 1), (1, 8, 2), (2, 5, 5), (3, 0, 2), (17, 4, 1), (131, 7, 7), (1000, 9, 3)])
@pytest.mark.parametrize("dtype", ["fp8_e4m3", "int8_per_token_head", "int4_per_token_head"])
def test_sizes(cuda_device, dtype, T, Hq, Hkv):
    c = Case(dtype, T, Hq, Hkv, 128, 128, False, T + Hq)
    if Hq:
        c.check(c.run(cuda_device))
        return
    # keys and values only
    qkv, row = c.qkv.to(cuda_device), kvq().cache_row_bytes(dtype, 128)
    c.kc = Guarded((c.blocks, c.block, Hkv, row), torch.uint8, FILL, cuda_device)
    c.vc = Guarded((c.blocks, c.block, Hkv, row), torch.uint8, FILL, cuda_device)
    kvq().rotary_and_cache(None, qkv[:, :Hkv], qkv[:, Hkv:], torch.from_numpy(c.positions).to(cuda_device),
                           torch.from_numpy(c.table).to(cuda_device), None, c.kc.t, c.vc.t,
                           torch.from_numpy(c.slots).to(cuda_device), dtype, False, c.k_scale, c.v_scale)
    c.check(np.zeros((T, 0, 128), np.int16))


def test_no_tokens(cuda_device):
    e = lambda *n, dtype=torch.bfloat16: torch.empty(n, dtype=dtype, device=cuda_device)  # noqa: E731
    kvq().rotary_and_cache(e(0, 4, 128), e(0, 2, 128), e(0, 2, 128), e(0, dtype=torch.int64),
                           e(4, 64, dtype=torch.float32), e(0, 4, 128), e(1, 16, 2, 144, dtype=torch.uint8),
                           e(1, 16, 2, 144, dtype=torch.uint8), e(0, dtype=torch.int64), "int8_per_token_head")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("scale", [1.0, 0.05, 2.0 ** -20, 2.0 ** -125, 3.0e37])
def test_every_bf16_value_is_coded_as_the_writer_codes_it(cuda_device, dtype, scale):
    """Cosines 1 and sines 0 leave the keys as they are: the bytes are
    reshape_and_cache's, for every finite bf16 value (ties, subnormals, the
    largest), in rows of values of all sizes and of one size."""
    bits = np.arange(65536, dtype=np.uint32)
    pats = bits[((bits >> 7) & 0xFF) != 0xFF].astype(np.uint16)
    pats = pats[(pats & 0x7FFF) != 0]   # (0 s added to -0 gives +0)
    rng = np.random.default_rng(3)
    D, H = 128, 2
    x = np.concatenate([np.sort(pats), rng.permutation(pats)])
    T = x.size // (H * D)
    key = torch.from_numpy(x[:T * H * D].view(np.int16).copy()).view(torch.bfloat16).view(T, H, D).to(cuda_device)
    value = key.flip(0).contiguous()
    table = torch.cat((torch.ones(4, 64), torch.zeros(4, 64)), 1).to(cuda_device)
    # (values that the sine's product would make NaN of: none, 0 times finite is 0)
    row = kvq().cache_row_bytes(dtype, D)
    caches = [torch.full((T // 16 + 1, 16, H, row), FILL, dtype=torch.uint8, device=cuda_device) for _ in range(4)]
    slots = torch.arange(T, device=cuda_device)
    kvq().reshape_and_cache(key, value, caches[0], caches[1], slots, dtype, scale, scale)
    kvq().rotary_and_cache(None, key, value, slots % 4, table, None, caches[2], caches[3], slots, dtype, False,
                           scale, scale)
    assert torch.equal(caches[0], caches[2])
    assert torch.equal(caches[1], caches[3])


@pytest.mark.parametrize("dtype", ["int8_per_token_head", "fp8_per_token_head", "fp8_e5m2_per_token_head",
                                   "int4_per_token_head"])
def test_special_rows(cuda_device, dtype):
    """Zero rows, rows of one value, subnormal rows, rows near the largest
    finite value, rows where a group is far smaller than the rest."""
    c = Case(dtype, 8, 2, 2, 128, 128, False, 5)
    x = c.qkv
    x[0] = 0.0
    x[1] = 3.0
    x[2] = x[2] * 2.0 ** -130
    x[3] = torch.sign(x[3]) * 1.5e38
    x[4, :, 32:] *= 2.0 ** -12
    x[5, :, 1:] = 0.0
    x[6] = x[6] * 2.0 ** -118
    c.positions[3] = 0   # (rotated values stay finite)
    c.check(c.run(cuda_device))


def test_caches_beyond_4_gib(cuda_device):
    D, H, row = 64, 8, kvq().cache_row_bytes("int8_per_token_head", 64)
    blocks = (1 << 32) // (16 * H * row) + 40
    kc = torch.empty((blocks, 16, H, row), dtype=torch.uint8, device=cuda_device)
    vc = torch.empty_like(kc)
    c = Case("int8_per_token_head", 5, 8, H, D, 64, False, 1)
    slots = torch.tensor([blocks * 16 - 1, 3, blocks * 16 - 20, (1 << 32) // (H * row) + 1, 0], device=cuda_device)
    for t in (kc, vc):
        t.view(-1, H, row)[slots] = 0
    qkv, out = c.qkv.to(cuda_device), torch.empty((5, 8, D), dtype=torch.bfloat16, device=cuda_device)
    kvq().rotary_and_cache(qkv[:, :8], qkv[:, 8:16], qkv[:, 16:], torch.from_numpy(c.positions).to(cuda_device),
                           torch.from_numpy(c.table).to(cuda_device), out, kc, vc, slots, "int8_per_token_head")
    x = c.qkv.double().numpy()
    want = R.rows("int8_per_token_head", R.rotate(x[:, 8:16], c.table, c.positions, False), 1.0)
    assert np.array_equal(kc.view(-1, H, row)[slots].cpu().numpy(), want)
    assert np.array_equal(vc.view(-1, H, row)[slots].cpu().numpy(), R.rows("int8_per_token_head", x[:, 16:], 1.0))


def test_on_another_stream_and_replayed(cuda_device):
    """Captured once, replayed with other rows, positions and slots in place."""
    s = torch.cuda.Stream()
    c = Case("fp8_per_token_head", 40, 8, 2, 128, 64, True, 21)
    got = c.run(cuda_device, stream=s)
    c.check(got)
    qkv, pos, table, slots = c.keep
    call = lambda: kvq().rotary_and_cache(  # noqa: E731
        qkv[:, :8], qkv[:, 8:10], qkv[:, 10:], pos, table, c.out.t, c.kc.t, c.vc.t, slots, c.dtype, True)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for seed in (22, 23):
        d = Case("fp8_per_token_head", 40, 8, 2, 128, 64, True, seed)
        c.qkv, c.positions, c.slots = d.qkv, d.positions, d.slots
        qkv.copy_(d.qkv)
        pos.copy_(torch.from_numpy(d.positions))
        slots.copy_(torch.from_numpy(d.slots))
        c.kc.t.fill_(FILL)
        c.vc.t.fill_(FILL)
        graph.replay()
        torch.cuda.synchronize()
        c.check(c.out.t.cpu().view(torch.int16).numpy())


@pytest.mark.parametrize("dtype", ["auto", "int8_per_token_head", "int4_per_token_head"])
def test_large_batches_are_stored_as_small_ones(cuda_device, dtype):
    """A batch of more than 64 MB of rows against its two halves, bit for bit."""
    T, Hq, H, D = 6001, 40, 8, 128
    g = torch.Generator(device=cuda_device).manual_seed(4)
    qkv = torch.randn((T, Hq + 2 * H, D), generator=g, device=cuda_device).to(torch.bfloat16)
    assert qkv.numel() * 2 > 64 << 20 and qkv.numel() < 64 << 20
    pos = torch.randint(0, 3000, (T,), generator=g, device=cuda_device)
    table = torch.from_numpy(R.cos_sin_table(3000, D)).to(cuda_device)
    slots = torch.randperm(T + 15, generator=g, device=cuda_device)[:T]
    slots[::97] = -1
    row = kvq().cache_row_bytes(dtype, D)
    got = []
    for parts in ([(0, T)], [(0, 3000), (3000, T)]):
        kc, vc = (torch.full((T // 16 + 1, 16, H, row), FILL, dtype=torch.uint8, device=cuda_device) for _ in range(2))
        out = torch.full((T, Hq, D), float("nan"), dtype=torch.bfloat16, device=cuda_device)
        for a, b in parts:
            x = qkv[a:b]
            kvq().rotary_and_cache(x[:, :Hq], x[:, Hq:Hq + H], x[:, Hq + H:], pos[a:b], table, out[a:b], kc, vc,
                                   slots[a:b], dtype)
        got.append((kc, vc, out.view(torch.int16)))
    assert all(torch.equal(a, b) for a, b in zip(*got))
    assert not torch.isnan(out).any()
