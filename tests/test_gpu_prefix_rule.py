"""A batch of 4-bit rows on both sides of the plan's rule: sharing has to save 18 MB
of cache reads."""
import pytest

from _shared import SharedRun, compare, shared_workload
from int8_kv_cache_reshape_gb300 import kvq

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("requests,D,Hq,Hkv", [(58, 128, 16, 8), (59, 128, 16, 8), (57, 256, 8, 4), (58, 256, 8, 4)])
def test_a_4_bit_batch_shared_by_the_rule(cuda_device, monkeypatch, requests, D, Hq, Hkv):
    monkeypatch.delenv("KVQ_PREFIX_MIN_BYTES", raising=False)
    dtype, P = "int4_per_token_head", 288 if D == 256 else 256
    saved = (requests - 1) * P * Hkv * 2 * kvq.cache_row_bytes(dtype, D)
    shared = requests if saved >= 18 << 20 else 0
    assert abs(saved - (18 << 20)) < 1 << 19   # (one request or so from the limit)
    wl = shared_workload([P], [0] * requests, [1 + 5 * r % 60 for r in range(requests)], [1] * requests, Hq, Hkv, D, 16,
                         dtype, 80 + requests)
    g = SharedRun(wl).write_cache().attention()
    assert g.rect["num_shared_requests"] == shared and (g.rect["num_units"] > 0) == (shared > 0)
    compare(g, f"{requests} requests")
