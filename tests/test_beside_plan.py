"""The plan of a batch that shares a prefix, where the decode is long: cut for the
SMs that the units leave, or behind short units.  (Host plans; without a device they are
made for 152 SMs.)"""
import numpy as np
import pytest

from int8_kv_cache_reshape_gb300 import kvq

SMS = 152


@pytest.mark.parametrize("dtype,warps", [("int8_per_token_head", 16), ("auto", 12)])
@pytest.mark.parametrize("R,P,own,sharers", [(64, 8192, 100, 2), (32, 8192, 8000, 8), (128, 8192, 1000, 2)])
def test_no_decode_behind_long_units(dtype, warps, R, P, own, sharers):
    """A decode on all SMs beside units has CTAs that wait for a unit and then take as
    long as all others: only units of up to 8 of the prefix's 64 KV tiles may be ahead of
    one (warps: of an SM at 32 / 8 heads of 128)."""
    lens = [P + own] * R
    of = [0 if r < sharers else -1 for r in range(R)]
    s = kvq.get_shared_prefix_metadata(R, 32, 8, 128, lens, list(range(R + 1)), [P], of, 0, dtype)
    units = s.rect_info()["num_units"]
    assert 0 < units < SMS
    assert s.info()["num_decode_warps"] <= warps * (SMS - units) or units >= 8 * 64 // 8
    w = kvq.get_scheduler_metadata(R, 32, 8, 128, np.array(lens, np.int32), np.arange(R + 1, dtype=np.int32), True, 0, dtype)
    assert w.info()["num_decode_warps"] == warps * SMS
