"""Rows of the pools that no query may see hold bytes that are NaN in every
format (0xFF: NaN fp8 codes and bf16 values, multipliers out of range, NaN
scales): behind the last key, before the first one that a window leaves, and in
the block that stands in for one that is missing from the table."""
import numpy as np
import pytest
import torch

from _shared import CrossRun, SharedRun, compare, shared_workload
from int8_kv_cache_reshape_gb300 import workloads as W

pytestmark = pytest.mark.gpu

DTYPES = ["auto", "fp8_e4m3", "fp8_e5m2", "int8_per_token_head", "fp8_per_token_head",
          "fp8_e5m2_per_token_head", "int4_per_token_head"]
HEADS = [(64, 8, 2), (128, 8, 2), (256, 4, 1)]


@pytest.fixture(autouse=True)
def share_everything(monkeypatch):
    """4-bit batches as small as these would not be shared."""
    monkeypatch.setenv("KVQ_PREFIX_MIN_BYTES", "0")


def _poisoned(g, wl):
    """The run's pools 0xFF wherever no listed token is stored."""
    for c in (g.kc, g.vc):
        c.fill_(0xFF)
    return g.write_cache()


def _cross(new, lens, Hq, Hkv, D, dtype, seed):
    return W.custom("cross", new, lens, Hq, Hkv, D, 16, dtype, seed, causal=False, extra_blocks=2,
                    token_scale_range=(0.2, 5.0) if "per_token" in dtype else None)


@pytest.mark.parametrize("tiles", [1, 100])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("D,Hq,Hkv", HEADS)
def test_behind_an_encoders_last_key(cuda_device, monkeypatch, tiles, dtype, D, Hq, Hkv):
    """Last chunks and tiles with 1 to 15 keys, on the units (20 rows and more a
    kv head) and on the split-KV decode (4 to 16)."""
    monkeypatch.setenv("KVQ_RECT_TILES", str(tiles))
    lens = [1, 9, 333, 50, 127, 190, 7, 75, 401]
    wl = _cross([5, 40, 33, 90, 5, 6, 1, 2, 4], lens, Hq, Hkv, D, dtype, 60 + D)
    g = _poisoned(CrossRun(wl), wl).attention()
    assert g.rect["num_units"] > 0 and g.sched_info["num_chunks"] > 0
    compare(g, f"{dtype} {D}")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("D,Hq,Hkv", HEADS)
def test_before_a_windows_first_key(cuda_device, dtype, D, Hq, Hkv):
    """A prefix of which no request sees the first keys, which end inside a chunk."""
    own = [40, 13, 77, 5, 60, 29]
    wl = shared_workload([333], [0] * 6, own, [1] * 6, Hq, Hkv, D, 16, dtype, 61, window=150)
    unseen = min(L - 1 - 149 for L in wl.seq_lens)
    assert unseen % 16 and unseen > 64
    wl.slot_mapping[wl.token_pos < unseen] = -1
    g = _poisoned(SharedRun(wl), wl).attention()
    assert g.rect["num_shared_requests"] == 6
    compare(g, f"{dtype} {D}")


def _without_block_0(wl):
    """The workload with its block 0 moved to a block of no request."""
    live = [wl.block_table[r, :-(-L // wl.block_size)] for r, L in enumerate(wl.seq_lens)]
    spare = sorted(set(range(wl.num_blocks)) - set(torch.cat(live).tolist()))[-1]
    wl.block_table[wl.block_table == 0] = spare
    at = (wl.slot_mapping >= 0) & (wl.slot_mapping < wl.block_size)
    wl.slot_mapping[at] += spare * wl.block_size
    return wl


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("D,Hq,Hkv", HEADS)
def test_missing_blocks(cuda_device, dtype, D, Hq, Hkv):
    """Requests whose last blocks are missing give what they give without them."""
    lens, cut = [320, 96, 480, 200], [16 * 15, 16 * 4, 16 * 27, 16 * 10]
    wl = _without_block_0(_cross([40, 5, 90, 1], lens, Hq, Hkv, D, dtype, 62))
    for r, n in enumerate(cut):
        wl.block_table[r, n // 16:] = -1 if r % 2 else wl.num_blocks + 3
        wl.slot_mapping[(wl.token_req == r) & (wl.token_pos >= n)] = -1
    g = _poisoned(CrossRun(wl), wl).attention()
    assert bool((g.kc[0] == 0xFF).all()) and np.isfinite(g.out_f32()).all()
    keep = wl.token_pos < torch.tensor(cut)[wl.token_req.long()]
    short = _cross([40, 5, 90, 1], cut, Hq, Hkv, D, dtype, 62)
    short.q, short.block_table, short.num_blocks = wl.q, wl.block_table, wl.num_blocks
    short.key, short.value, short.slot_mapping = wl.key[keep], wl.value[keep], wl.slot_mapping[keep]
    short.token_req, short.token_pos = wl.token_req[keep], wl.token_pos[keep]
    short.k_scale, short.v_scale, short.sm_scale = wl.k_scale, wl.v_scale, wl.sm_scale
    h = CrossRun(short).write_cache()
    h.attention()
    compare(h, f"{dtype} {D}")
    h.out.copy_(g.out)
    compare(h, f"{dtype} {D}, blocks missing")
