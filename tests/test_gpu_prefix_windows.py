"""Windowed batches that share a prefix, whose requests no longer hold the blocks
behind their own windows: a server that gives such blocks back leaves -1, or the
id of a block that now holds other rows, in their table entries."""
import pytest
import torch

from _shared import SharedRun, compare, shared_workload

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def share_everything(monkeypatch):
    """4-bit batches as small as these would not be shared."""
    monkeypatch.setenv("KVQ_PREFIX_MIN_BYTES", "0")


def _released(wl, entry):
    """The table with every entry that lies wholly behind its request's window
    replaced; returns how many of the prefix's entries that are."""
    n = 0
    for r, (L, Q) in enumerate(zip(wl.seq_lens, wl.query_lens)):
        gone = max(0, L - Q - wl.window + 1) // wl.block_size
        wl.block_table[r, :gone] = entry
        n += min(gone, wl.prefix_lens[wl.of[r]] // wl.block_size) if wl.of[r] >= 0 else 0
    return n


@pytest.mark.parametrize("order", ["longest first", "shortest first", "mixed"])
@pytest.mark.parametrize("entry", ["-1", "a block of other rows"])
@pytest.mark.parametrize("dtype,D", [("int8_per_token_head", 128), ("fp8_e4m3", 64), ("auto", 256),
                                     ("int4_per_token_head", 128)])
def test_entries_behind_the_windows(cuda_device, order, entry, dtype, D):
    own = [139 - 17 * r for r in range(9)]
    if order == "shortest first":
        own.reverse()
    if order == "mixed":
        own = own[4:] + own[:4]
    wl = shared_workload([350], [0] * 9, own, [1, 2, 1, 1, 3, 1, 1, 1, 2], 8, 2, D, 16, dtype, 5, window=200)
    # (a block of no request, whose rows keep the pool's fill)
    spare = sorted(set(range(wl.num_blocks)) - set(wl.block_table.flatten().tolist()))[0]
    assert _released(wl, -1 if entry == "-1" else spare) > 9
    g = SharedRun(wl).write_cache().attention()
    assert g.rect["num_shared_requests"] == 9 and g.rect["num_units"] > 0
    compare(g, f"{dtype}, {order}")


@pytest.mark.parametrize("tiles", [1, 2, 100])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_row_tiles_of_their_own_windows(cuda_device, monkeypatch, tiles, D):
    """Two prefixes and several row tiles each, in which windows begin ever later
    or ever earlier; keys cut into units of one, two and all KV tiles."""
    monkeypatch.setenv("KVQ_RECT_TILES", str(tiles))
    R = 70
    of = [r % 2 for r in range(2 * R)]
    own = [1 + 4 * (r // 2) if r % 2 else 261 - 3 * (r // 2) for r in range(2 * R)]
    wl = shared_workload([700, 500], of, own, [1] * (2 * R), 8, 2, D, 32, "int8_per_token_head", 6, window=300)
    assert _released(wl, -1) > R
    g = SharedRun(wl).write_cache().attention()
    assert g.rect["num_shared_requests"] == 2 * R
    compare(g, f"{D}, {tiles} tiles a unit")


def test_results_do_not_depend_on_the_released_entries(cuda_device):
    """The same batch with whole tables and with released entries, bit for bit."""
    wl = shared_workload([600], [0] * 12, [220 - 18 * r for r in range(12)], [1] * 12, 8, 2, 128, 16, "fp8_e4m3", 7,
                         window=250)
    whole = SharedRun(wl).write_cache().attention().out.clone()
    assert _released(wl, -1) > 12
    assert torch.equal(SharedRun(wl).write_cache().attention().out, whole)
