"""Rotated queries that would be stored over the caches are refused before a launch
(calls that need no GPU), and no others are."""
import pytest
import torch

from int8_kv_cache_reshape_gb300 import kvq

A = 1 << 20
ROW = kvq.cache_row_bytes("int8_per_token_head", 128)
POOL = 4 * 16 * 2 * ROW      # bytes of a pool of 4 blocks of 16 slots, 2 heads
# arguments of kvq_rotary_and_cache by position (addresses that are never read): 5 tokens, 4 / 2 heads of 128
GOOD = dict(enumerate([A, 2 * A, 3 * A, 5, 512, 256, 256, 4, 2, 128, 4 * A, 5 * A, 9, 64, 0, 6 * A, 512, 7 * A, 8 * A, 4,
                       16, 9 * A, 3, 1.0, 1.0, None]))
LAST = 4 * 1024              # bytes to the last of five query rows
WIDE = 1 << 16               # bytes from row to row of a wide output


def _call(**changes):
    args = {**GOOD, **{int(k[1:]): v for k, v in changes.items()}}
    return kvq.lib.kvq_rotary_and_cache(*args.values())


@pytest.mark.parametrize("cache,at", [(17, 7 * A), (18, 8 * A)])
@pytest.mark.parametrize("offset", [0, 16, POOL - 16, -16, -LAST - 1024 + 16, -LAST])
def test_a_query_output_over_a_pool(cache, at, offset):
    """From the pool's first byte to its last, by the rows' first and their last."""
    assert _call(**{f"a{cache}": at, "a15": at + offset}) == kvq.E_INVALID_ARG


@pytest.mark.parametrize("offset", [16, POOL - 16, -16])
def test_queries_rotated_in_place_over_a_pool(offset):
    assert _call(a0=7 * A + offset, a15=7 * A + offset) == kvq.E_INVALID_ARG


@pytest.mark.parametrize("offset", [1024 - 16, WIDE - POOL + 16, 2 * WIDE, 4 * WIDE - 16, 4 * WIDE + 1008])
def test_a_pool_that_meets_a_row_of_a_wide_output(offset):
    assert _call(a15=16 * A, a16=WIDE // 2, a17=16 * A + offset) == kvq.E_INVALID_ARG


@pytest.mark.gpu
def test_pools_between_the_rows_of_a_wide_output(cuda_device):
    """Pools that begin where a row ends, end where the next begins or lie behind the
    last one meet none of them: the same rows and queries as in buffers of their own."""
    gen = torch.Generator().manual_seed(2)
    qkv = torch.randn((5, 8, 128), generator=gen).to(torch.bfloat16).to(cuda_device)
    table = torch.randn((9, 64), generator=gen).to(cuda_device)
    pos, slots = torch.arange(5, device=cuda_device), 3 + 7 * torch.arange(5, device=cuda_device)

    def rotate(out, kc, vc):
        kvq.rotary_and_cache(qkv[:, :4], qkv[:, 4:6], qkv[:, 6:], pos, table, out, kc, vc, slots, "int8_per_token_head")
        torch.cuda.synchronize()
        return out.clone(), kc.clone(), vc.clone()

    want = rotate(torch.zeros((5, 4, 128), dtype=torch.bfloat16, device=cuda_device),
                  *(torch.zeros((4, 16, 2, ROW), dtype=torch.uint8, device=cuda_device) for _ in range(2)))
    for k_at, v_at in ((1024, 2 * WIDE - POOL), (3 * WIDE + 5008, 4 * WIDE + 1024)):
        buf = torch.zeros(5 * WIDE, dtype=torch.uint8, device=cuda_device)
        out = buf.view(torch.bfloat16).as_strided((5, 4, 128), (WIDE // 2, 128, 1))
        got = rotate(out, *(buf[at:at + POOL].view(4, 16, 2, ROW) for at in (k_at, v_at)))
        assert all(torch.equal(a, b) for a, b in zip(got, want))
