"""Shared memory that a 4-bit schedule reports: that of the launch classes it
has tiles for (host only)."""
import numpy as np
import pytest

from int8_kv_cache_reshape_gb300 import kvq

# A decode CTA has rings of `stages` chunks (up to 8) of 32 tokens, K and V, of
# one group of heads a ring, 32 bytes of bookkeeping a stage and 1 KB to align
# them, within 212 KB.  8 heads of 128 (80-byte rows) are 8 warps: two groups
# of 16 warps for tiles of up to 8 rows, one of 12 above.
STAGE = 2 * 32 * 8 * 80
ROOM = 211 * 1024
CLASS = [2 * (ROOM // (2 * (STAGE + 32))) * (STAGE + 32) + 1024, (ROOM // (STAGE + 32)) * (STAGE + 32) + 1024]


def _info(ql, sl, heads_q):
    s = kvq.get_scheduler_metadata(len(sl), heads_q, 8, 128, np.array(sl, np.int32),
                                   np.concatenate([[0], np.cumsum(ql)]).astype(np.int32), True, 0,
                                   "int4_per_token_head")
    return s.info()


@pytest.mark.parametrize("ql,heads_q,want", [
    ([1, 1], 64, CLASS[0]),              # tiles of 8 rows
    ([1, 1], 128, CLASS[1]),             # of 16
    ([2, 1], 64, max(CLASS)),            # of both
    ([4], 32, CLASS[1]),
    ([300], 32, CLASS[0]),               # a prefill: no decode launch
])
def test_shared_memory_of_the_launched_classes(ql, heads_q, want):
    assert CLASS[0] != CLASS[1]
    info = _info(ql, [500] * len(ql), heads_q)
    assert info["decode_smem_bytes"] == want
