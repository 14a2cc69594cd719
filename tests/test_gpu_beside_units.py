"""The decode beside the units of a shared prefix: requests whose own contexts are
long.  Times are compared with those of the same batch planned without sharing."""
import numpy as np
import pytest
import torch

from int8_kv_cache_reshape_gb300 import kvq

pytestmark = pytest.mark.gpu

HQ, HKV, D, B = 32, 8, 128, 16


def _calls(dtype, P, own, new, sharers, device, HQ=HQ, HKV=HKV, D=D):
    """One batch planned with its prefix and without: (call, schedule) of each."""
    R = len(own)
    lens = np.array([P + n for n in own], np.int32)
    need = [-(-int(n) // B) for n in lens]
    gen = torch.Generator(device).manual_seed(1)
    shape = (sum(need), B, HKV, kvq.cache_row_bytes(dtype, D))
    if dtype == "auto":
        kc = torch.randn((*shape[:3], D), generator=gen, device=device).to(torch.bfloat16).view(torch.uint8)
    else:       # (rows of one scale, 2^-6; 4-bit ones of multipliers of 50)
        kc = torch.randint(0, 100, shape, generator=gen, dtype=torch.uint8, device=device)
        at = D // 2 if dtype == "int4_per_token_head" else D
        kc[..., at:at + 4] = torch.tensor([0, 0, 128, 60], dtype=torch.uint8, device=device)
        kc[..., at + 4:at + 12] = 50
    vc = kc.flip(0)
    bt = torch.zeros((R, max(need)), dtype=torch.int32, device=device)
    blocks = torch.randperm(sum(need), generator=gen, device=device).to(torch.int32)
    for r, n in enumerate(need):
        bt[r, :n] = blocks[sum(need[:r]):sum(need[:r + 1])]
    bt[:sharers, :P // B] = bt[0, :P // B]
    starts = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    q = torch.randn((int(starts[-1]), HQ, D), generator=gen, device=device).to(torch.bfloat16)
    qsl, sl = torch.from_numpy(starts).to(device), torch.from_numpy(lens).to(device)
    of = [0 if r < sharers else -1 for r in range(R)]
    runs = []
    for s in (kvq.get_shared_prefix_metadata(R, HQ, HKV, D, lens, starts, [P], of, 0, dtype),
              kvq.get_scheduler_metadata(R, HQ, HKV, D, lens, starts, True, 0, dtype)):
        out = torch.full_like(q, float("nan"))
        ws = torch.empty(max(256, s.workspace_bytes), dtype=torch.uint8, device=device)
        call = kvq.prepare_attention_with_kv_cache(s, q, kc, vc, qsl, sl, bt, D ** -0.5, True, 0, 0.0, 1.0, 1.0, out, ws,
                                                   dtype, HKV)
        runs.append((call, s, out, (ws, q, kc, vc, qsl, sl, bt)))
    return runs


def _us(call, n=20):
    times = []
    for _ in range(5):
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        call()
        a.record()
        for _ in range(n):
            call()
        b.record()
        torch.cuda.synchronize()
        times.append(1e3 * a.elapsed_time(b) / n)
    return sorted(times)[2]


def _compare(runs):
    """Times of the shared and the unshared call, whose results agree."""
    (a, sa, oa, _), (b, sb, ob, _) = runs
    assert sa.rect_info()["num_units"] > 0 and sb.rect_info()["num_units"] == 0
    times = _us(a), _us(b)
    for _, s, _, _ in runs:
        s.check_device()
        s.close()
    # both are within half a bf16 step (2^-9 of the value) plus their fp32 sums of the exact result
    x, y = oa.double(), ob.double()
    assert (x - y).abs().max() <= 2.0 ** -7 * y.abs().max()
    return times


@pytest.mark.parametrize("dtype,P,own,new,sharers", [
    ("int8_per_token_head", 32, [8192] * 64, [1] * 64, 2),      # few units, a long decode on all SMs
    ("int8_per_token_head", 2048, [8192] * 64, [1] * 64, 64),
    ("auto", 32, [3000] * 64, [1] * 64, 2),
    ("int8_per_token_head", 2048, [2048] * 64, [1, 3] * 32, 64),  # both row classes
])
def test_a_long_decode_beside_short_units(cuda_device, dtype, P, own, new, sharers):
    """Sharing saves reads here or next to none; it must not cost half as much again
    (CTAs behind a unit on its SM took 2.4 times as long as the others: 1.8 to 2.5 times
    the unshared call)."""
    shared, unshared = _compare(_calls(dtype, P, own, new, sharers, cuda_device))
    assert shared <= 1.5 * unshared, f"{shared:.0f} us with the prefix shared, {unshared:.0f} us without"


@pytest.mark.parametrize("D,HQ,HKV,P,own,sharers", [(256, 16, 4, 2048, 1000, 16), (256, 16, 4, 8192, 8000, 16),
                                                    (64, 8, 2, 4096, 2000, 64)])
def test_a_4_bit_decode_on_the_sms_that_units_leave(cuda_device, D, HQ, HKV, P, own, sharers):
    """It is cut for those SMs: with a CTA for each SM of the device the last ones
    waited for whole units (1.3 to 1.4 times the time)."""
    runs = _calls("int4_per_token_head", P, [own // 2 + 16 * r for r in range(64)], [1] * 64, sharers, cuda_device, HQ, HKV, D)
    shared, unshared = _compare(runs)
    assert shared <= 1.15 * unshared, f"{shared:.0f} us with the prefix shared, {unshared:.0f} us without"


def test_both_classes_of_a_4_bit_decode(cuda_device):
    """Tiles of 4 and of 12 rows a kv head, each class cut for its part of the SMs left:
    one class after the other took 1.3 times the unshared call, 1.8 times both together."""
    runs = _calls("int4_per_token_head", 2048, [2048] * 64, [1, 3] * 32, 64, cuda_device)
    shared, unshared = _compare(runs)
    assert shared <= unshared, f"{shared:.0f} us with the prefix shared, {unshared:.0f} us without"


@pytest.mark.parametrize("dtype,R,P,own,sharers", [
    ("int8_per_token_head", 64, 8192, 100, 2), ("auto", 8, 8192, 8000, 2), ("auto", 8, 2048, 1000, 2),
    ("int4_per_token_head", 64, 8192, 8000, 16)])
def test_few_requests_behind_a_long_prefix(cuda_device, dtype, R, P, own, sharers):
    """Long units beside a long decode of requests without the prefix, or with long
    contexts of their own: 1.6 to 1.9 times the unshared call where the decode was cut for
    all SMs, or the units too long."""
    shared, unshared = _compare(_calls(dtype, P, [own + 16 * (r % 3) for r in range(R)], [1] * R, sharers, cuda_device))
    assert shared <= 1.3 * unshared, f"{shared:.0f} us with the prefix shared, {unshared:.0f} us without"
