"""build_block_tables over lengths that do not fit: starts that decrease, and
requests left out of batches that span several CTAs (1,024 tokens each) and
several windows of requests (1,024 each).  Whole numbers: equality."""
import numpy as np
import pytest
import torch

from _harness import Guarded, kvq
from test_gpu_gather_tables import _run_tables, _tables_case

pytestmark = pytest.mark.gpu


def _starts(R, kind):
    """Starts of R requests that decrease once (or often)."""
    qsl = np.arange(R + 1) * 3
    if kind == "first":
        qsl[1:] -= 5
    elif kind == "middle":
        qsl[R // 2 + 1:] -= 7
    elif kind == "last":
        qsl[R] -= 4
    else:
        qsl = qsl[::-1].copy()
    return qsl.astype(np.int32)


@pytest.mark.parametrize("R", [1, 2, 3, 700, 1024, 1025, 3000])
@pytest.mark.parametrize("kind", ["first", "middle", "last", "all"])
@pytest.mark.parametrize("alias", [False, True])
def test_decreasing_starts_leave_the_step_out(cuda_device, R, kind, alias):
    dev, block, width = cuda_device, 16, 4
    qsl = _starts(R, kind)
    assert (np.diff(qsl) < 0).any()
    i32 = lambda v: torch.tensor(np.asarray(v, np.int32), device=dev)  # noqa: E731
    rng = np.random.default_rng(R)
    table = Guarded((R, width), torch.int32, 0, dev)
    old = torch.from_numpy(rng.integers(0, 4 * R, (R, width)).astype(np.int32))
    table.t.copy_(old)
    slots = Guarded((3 * R + 5,), torch.int64, 123, dev)
    free = i32(rng.permutation(4 * R))
    count = i32([4 * R])
    left = count if alias else i32([-9])
    status = i32([0] * 4)
    for _ in range(2):
        kvq().build_block_tables(i32(qsl), i32(rng.integers(3, 60, R)), free, count, table.t, slots.t, block, 4 * R,
                                 left, status)
        torch.cuda.synchronize()
        table.check("block table")
        slots.check("slot mapping")
        assert (slots.t == -1).all()
        assert torch.equal(table.t.cpu(), old)
        assert int(left) == 4 * R
        assert status.cpu().tolist()[:3] == [0, R, 0]


def test_a_step_after_one_left_out(cuda_device):
    """The status word is ready for the next call, and requests that share a
    start (no new tokens) do not count as a decrease."""
    dev = cuda_device
    i32 = lambda v: torch.tensor(np.asarray(v, np.int32), device=dev)  # noqa: E731
    free, count, status = i32([5, 6, 7]), i32([3]), i32([0] * 4)
    table = torch.full((3, 2), -1, dtype=torch.int32, device=dev)
    slots = torch.zeros(4, dtype=torch.int64, device=dev)
    for qsl, want, left, bad in (([0, 3, 1, 4], [-1] * 4, 3, 3), ([0, 2, 2, 3], [7 * 16, 7 * 16 + 1, 6 * 16, -1], 1, 0)):
        kvq().build_block_tables(i32(qsl), i32([2, 0, 1]), free, count, table, slots, 16, 8, count, status)
        assert slots.cpu().tolist() == want
        assert int(count) == left and status.cpu().tolist()[:3] == [0, bad, 0]


@pytest.mark.parametrize("R,max_q", [(1500, 3), (2500, 1), (5000, 2), (900, 40), (1024, 9), (1025, 9)])
@pytest.mark.parametrize("alias", [False, True])
def test_requests_left_out_of_large_batches(cuda_device, R, max_q, alias):
    """More new tokens than keys, or more blocks than the table has columns,
    scattered over the batch and in runs at its start, its end and on both
    sides of a window's border."""
    rng = np.random.default_rng(R + max_q)
    sl = rng.integers(1, 90, R).tolist()
    ql = [int(rng.integers(0, min(L, max_q) + 1)) for L in sl]
    odd = set(rng.choice(R, R // 7, replace=False).tolist()) | {0, 1, R - 1} | set(range(min(R, 1030) - 9, min(R, 1030)))
    for r in odd:
        if r % 2:
            ql[r] = max(1, ql[r])
            sl[r] = ql[r] - 1              # (a left-out request's tokens still take their places)
        else:
            ql[r], sl[r] = max(1, ql[r]), 400
    c = _tables_case(rng, ql, sl, 16, spare=R, width=6, pad=77)
    assert _run_tables(c, cuda_device, alias)[4] == len(odd)


@pytest.mark.parametrize("R", [40, 1600])
def test_tokens_past_the_buffer_of_a_large_batch(cuda_device, R):
    """The requests whose tokens do not fit the slot mapping are left out."""
    rng = np.random.default_rng(R)
    sl = rng.integers(1, 90, R).tolist()
    ql = [int(rng.integers(0, min(L, 50) + 1)) for L in sl]
    ql[-1] = 1
    c = _tables_case(rng, ql, sl, 16, spare=9)
    c["slots"] = sum(ql[: R - R // 4]) + 1
    assert _run_tables(c, cuda_device)[4] >= 1
