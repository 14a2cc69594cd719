"""4-bit attention at the smallest value scales, over many keys: multiplying
the values by a power of two multiplies the outputs by it, bit for bit, as
long as every stored number (row scales, outputs) is a normal one.

The normaliser is driven to 2^31 and more: the first 128 keys score 0 and set
the softmax's reference, all others score just short of moving it (2^8 above
the first, weights of 2^14).
"""
import math

import numpy as np
import pytest
import torch

from _harness import kvq

pytestmark = pytest.mark.gpu

DT = "int4_per_token_head"
L = 1 << 18
B = 16


def _run(D, Q, heads_q, mul):
    dev = torch.device("cuda:0")
    g = torch.Generator(dev)
    g.manual_seed(D + Q)
    key = torch.full((L, 1, D), 5.4 / math.sqrt(D), device=dev).bfloat16()   # z = 5.4: 2^7.8
    key[:128] = 0
    dims = 0.5 + 0.45 * torch.rand((1, 1, D), generator=g, device=dev)
    value = (dims * (1.0 + 0.05 * torch.rand((L, 1, D), generator=g, device=dev))).bfloat16()
    value = (value.float() * mul).bfloat16()                                # (exact: no subnormal)
    k = kvq()
    row = k.cache_row_bytes(DT, D)
    kc = torch.zeros((L // B, B, 1, row), dtype=torch.uint8, device=dev)
    vc = torch.zeros_like(kc)
    slots = torch.arange(L, device=dev)
    k.reshape_and_cache(key, value, kc, vc, slots, DT)
    q = torch.ones((Q, heads_q, D), dtype=torch.bfloat16, device=dev)
    out = torch.full_like(q, float("nan"))
    qsl, sl = np.array([0, Q], np.int32), np.array([L], np.int32)
    s = k.get_scheduler_metadata(1, heads_q, 1, D, sl, qsl, True, 0, DT)
    ws = torch.zeros(max(256, s.workspace_bytes), dtype=torch.uint8, device=dev)
    table = torch.arange(L // B, dtype=torch.int32, device=dev)[None]
    k.attention_with_kv_cache(s, q, kc, vc, torch.from_numpy(qsl).to(dev), torch.from_numpy(sl).to(dev), table,
                              1.0 / math.sqrt(D), True, 0, 0.0, 1.0, 1.0, out, ws, DT, 1)
    torch.cuda.synchronize()
    s.check_device()
    return out.double(), s.info()


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("Q,heads_q", [(1, 4), (2, 7), (40, 8)])
def test_outputs_follow_the_values_power_of_two(cuda_device, monkeypatch, D, Q, heads_q):
    monkeypatch.setenv("KVQ_DECODE_WARPS", "1")      # (a tile of one piece: one normaliser over all keys)
    want, info = _run(D, Q, heads_q, 1.0)
    assert info["num_merge_items"] == 0
    assert (info["num_prefill_tiles"] > 0) == (Q == 40)
    assert (want > 0.4).all() and (want < 1.1).all()
    # rows' maxima of 2^-116 and more: scales of 2^-125.8 and more
    for e in (-60, -115):
        got, _ = _run(D, Q, heads_q, 2.0 ** e)
        assert torch.equal(got * 2.0 ** -e, want)
