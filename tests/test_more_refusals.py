"""What rotary_and_cache and the shared-prefix and cross-attention plans refuse,
in the binding and in the library.  No call here reaches a kernel: every one
is refused before a launch, or only marshals or plans, so no GPU is needed."""
import ctypes

import numpy as np
import pytest
import torch

from int8_kv_cache_reshape_gb300 import kvq


def _tensors(T=5, Hq=4, H=2, D=128, R=64, dtype="int8_per_token_head", **kw):
    bf = lambda *n: torch.zeros(n, dtype=torch.bfloat16)  # noqa: E731
    row = kvq.cache_row_bytes(dtype, D)
    a = dict(query=bf(T, Hq, D), key=bf(T, H, D), value=bf(T, H, D), positions=torch.zeros(T, dtype=torch.int64),
             cos_sin=torch.zeros(9, R), query_out=bf(T, Hq, D), key_cache=torch.zeros((4, 16, H, row), dtype=torch.uint8),
             value_cache=torch.zeros((4, 16, H, row), dtype=torch.uint8),
             slot_mapping=torch.zeros(T, dtype=torch.int64), kv_cache_dtype=dtype, stream=0)
    a.update(kw)
    return a


@pytest.mark.parametrize("dtype", list(kvq.DTYPES))
def test_prepared_rotary(dtype):
    for D in (64, 128, 256):
        kvq.prepare_rotary_and_cache(**_tensors(D=D, dtype=dtype))
    # rows of one projection, a single token (which has no stride), no queries, none at all
    qkv = torch.zeros((5, 8, 128), dtype=torch.bfloat16)
    p = kvq.prepare_rotary_and_cache(**_tensors(dtype=dtype, query=qkv[:, :4], key=qkv[:, 4:6], value=qkv[:, 6:]))
    assert [p.args[i].value for i in (4, 5, 6, 16)] == [1024, 1024, 1024, 512]
    one = kvq.prepare_rotary_and_cache(**_tensors(T=1, dtype=dtype, query=qkv[:1, :4].as_strided((1, 4, 128), (3, 128, 1))))
    assert one.args[4].value == 512
    kvq.prepare_rotary_and_cache(**_tensors(dtype=dtype, query=None, query_out=None))
    kvq.prepare_rotary_and_cache(**_tensors(T=0, dtype=dtype))


@pytest.mark.parametrize("name,make", [
    ("query", lambda t: None),
    ("query_out", lambda t: None),
    ("query", lambda t: t.zeros((5, 4, 128))),
    ("query", lambda t: t.zeros((4, 4, 128), dtype=t.bfloat16)),
    ("query_out", lambda t: t.zeros((5, 2, 128), dtype=t.bfloat16)),
    ("key", lambda t: t.zeros((5, 4, 128), dtype=t.bfloat16)[:, ::2]),
    ("key", lambda t: t.zeros((5, 2, 256), dtype=t.bfloat16)[..., ::2]),
    ("value", lambda t: t.zeros((5, 2, 64), dtype=t.bfloat16)),
    ("value", lambda t: t.zeros((5, 2, 128), dtype=t.float16)),
    ("positions", lambda t: t.zeros(5, dtype=t.int32)),
    ("positions", lambda t: t.zeros(10, dtype=t.int64)[::2]),
    ("positions", lambda t: t.zeros(4, dtype=t.int64)),
    ("slot_mapping", lambda t: t.zeros(6, dtype=t.int64)),
    ("slot_mapping", lambda t: t.zeros(5, dtype=t.int32)),
    ("cos_sin", lambda t: t.zeros((9, 64), dtype=t.bfloat16)),
    ("cos_sin", lambda t: t.zeros((9, 128))[:, :64]),
    ("cos_sin", lambda t: t.zeros(64)),
    ("key_cache", lambda t: t.zeros((4, 16, 2, 128), dtype=t.uint8)),
    ("key_cache", lambda t: t.zeros((5, 16, 2, 144), dtype=t.uint8)),
    ("value_cache", lambda t: t.zeros((4, 16, 3, 144), dtype=t.uint8)),
    ("value_cache", lambda t: t.zeros((8, 16, 2, 144), dtype=t.uint8)[::2]),
])
def test_prepared_rotary_refusals(name, make):
    with pytest.raises(ValueError):
        kvq.prepare_rotary_and_cache(**_tensors(**{name: make(torch)}))


# arguments of kvq_rotary_and_cache by position (addresses that are never read)
A = 1 << 20
GOOD = [A, 2 * A, 3 * A, 5, 512, 256, 256, 4, 2, 128, 4 * A, 5 * A, 9, 64, 0, 6 * A, 512, 7 * A, 8 * A, 4, 16, 9 * A, 3,
        1.0, 1.0, None]


@pytest.mark.parametrize("changes,status", [
    ({3: -1}, kvq.E_INVALID_ARG), ({4: 504}, kvq.E_INVALID_ARG), ({4: 516}, kvq.E_INVALID_ARG),
    ({5: 255}, kvq.E_INVALID_ARG), ({6: 248}, kvq.E_INVALID_ARG), ({7: -1}, kvq.E_INVALID_ARG),
    ({8: 0}, kvq.E_INVALID_ARG), ({9: 96}, kvq.E_UNSUPPORTED), ({12: -1}, kvq.E_INVALID_ARG),
    ({12: 0}, kvq.E_INVALID_ARG), ({13: 0}, kvq.E_INVALID_ARG), ({13: 144}, kvq.E_INVALID_ARG),
    ({13: 24}, kvq.E_UNSUPPORTED), ({14: 2}, kvq.E_INVALID_ARG), ({16: 256}, kvq.E_INVALID_ARG),
    ({19: -1}, kvq.E_INVALID_ARG), ({20: 0}, kvq.E_INVALID_ARG), ({22: 7}, kvq.E_INVALID_ARG),
    ({22: 1, 23: 0.0}, kvq.E_INVALID_ARG), ({22: 2, 24: float("nan")}, kvq.E_INVALID_ARG),
    # addresses: missing, off their alignment
    *[({i: None}, kvq.E_INVALID_ARG) for i in (0, 1, 2, 10, 11, 15, 17, 18, 21)],
    *[({i: GOOD[i] + 8}, kvq.E_INVALID_ARG) for i in (0, 1, 2, 11, 15, 17, 18)],
    *[({i: GOOD[i] + 4}, kvq.E_INVALID_ARG) for i in (10, 21)],
    # queries written over queries that are still to be read
    ({15: A + 256}, kvq.E_INVALID_ARG), ({15: A, 16: 1024}, kvq.E_INVALID_ARG),
    ({4: 1024, 16: 1024, 15: A + 256}, kvq.E_INVALID_ARG), ({4: 1024, 16: 1024, 15: A - 512}, kvq.E_INVALID_ARG),
    # over keys or values: between their rows, over the last, a single token's
    ({15: 2 * A - 512}, kvq.E_INVALID_ARG), ({15: 3 * A + 4 * 512}, kvq.E_INVALID_ARG),
    ({16: 1024, 4: 1024, 5: 1024, 15: A + 1024, 1: A + 2048 - 16}, kvq.E_INVALID_ARG),
    ({3: 1, 15: 2 * A + 496}, kvq.E_INVALID_ARG),
    ({3: 1 << 31}, kvq.E_UNSUPPORTED), ({4: 1 << 31}, kvq.E_INVALID_ARG), ({6: 1 << 40}, kvq.E_INVALID_ARG),
])
def test_rotary_arguments(changes, status):
    args = list(GOOD)
    for i, v in changes.items():
        args[i] = v
    assert kvq.lib.kvq_rotary_and_cache(*args) == status


def test_rotary_without_tokens_is_no_call():
    assert kvq.lib.kvq_rotary_and_cache(None, None, None, 0, 0, 0, 0, 4, 2, 128, None, None, 0, 64, 0, None, 0, None, None,
                                        4, 16, None, 3, 1.0, 1.0, None) == kvq.OK


def _shared(lens=(40, 50), qsl=(0, 1, 2), prefixes=(16,), of=(0, 0), hq=8, hkv=2, d=128, window=0,
            dtype="int8_per_token_head"):
    return kvq.get_shared_prefix_metadata(len(of), hq, hkv, d, list(lens), list(qsl), list(prefixes), list(of), window, dtype)


@pytest.mark.parametrize("kw,status", [
    (dict(prefixes=(40,)), kvq.E_INVALID_ARG),       # beyond the first request's L - Q
    (dict(prefixes=(-1,)), kvq.E_INVALID_ARG),
    (dict(of=(0, 1)), kvq.E_INVALID_ARG),
    (dict(of=(0, -2)), kvq.E_INVALID_ARG),
    (dict(prefixes=(), of=(0, 0)), kvq.E_INVALID_ARG),
    (dict(lens=(40, -1)), kvq.E_INVALID_ARG),
    (dict(qsl=(0, 2, 1)), kvq.E_INVALID_ARG),
    (dict(qsl=(1, 2, 3)), kvq.E_INVALID_ARG),
    (dict(lens=(40, 1), qsl=(0, 1, 3), of=(0, -1)), kvq.E_INVALID_ARG),   # Q > L
    (dict(hq=7), kvq.E_UNSUPPORTED),
    (dict(d=96), kvq.E_UNSUPPORTED),
])
def test_shared_prefix_refusals(kw, status):
    with pytest.raises(kvq.KvqError) as e:
        _shared(**kw)
    assert e.value.status == status


@pytest.mark.parametrize("kw", [dict(lens=(40, 50, 60)), dict(qsl=(0, 1)), dict(of=(0, 0.5)), dict(prefixes=(2 ** 31,)),
                                dict(lens=(40, 2 ** 40))])
def test_shared_prefix_arrays(kw):
    with pytest.raises(ValueError):
        _shared(**kw)


def test_shared_prefix_plans_that_share_nothing():
    """No prefix, one member, prefixes below 32 keys, prompts, requests without
    queries, an empty batch: the plan of the batch without sharing."""
    for kw in (dict(of=(-1, -1)), dict(of=(0, -1)), dict(prefixes=(31,)), dict(prefixes=(0,)),
               dict(lens=(70, 90), qsl=(0, 30, 60), prefixes=(32,)), dict(qsl=(0, 0, 0), prefixes=(49,)),
               dict(lens=(), qsl=(0,), of=()), dict(prefixes=(), of=(-1, -1))):
        s = _shared(**kw)
        a = s.info()
        assert s.rect_info()["num_units"] == 0 and s.rect_info()["num_shared_requests"] == 0
        b = dict(lens=(40, 50), qsl=(0, 1, 2), of=(0, 0))
        b.update(kw)
        w = kvq.get_scheduler_metadata(len(b["of"]), 8, 2, 128, list(b["lens"]), list(b["qsl"]), True, 0,
                                       "int8_per_token_head")
        assert a["num_chunks"] == w.info()["num_chunks"] and a["num_prefill_tiles"] == w.info()["num_prefill_tiles"]


def test_shared_prefix_reads_each_key_once():
    """Chunks of the requests' own keys, and units whose partials the merge reads."""
    own, P = [5, 33, 1, 16, 700], 320
    s = _shared([P + n for n in own], range(6), [P], [0] * 5)
    assert s.rect_info()["num_shared_requests"] == 5 and s.rect_info()["shared_keys"] == 5 * P
    assert s.info()["num_chunks"] == 2 * sum(-(-n // 16) for n in own)   # (kv heads, chunks of 16)
    assert s.rect_info()["num_merge_items"] == 10
    # a window that reaches into the prefix for the shorter ones only
    w = _shared([P + n for n in own], range(6), [P], [0] * 5, window=64)
    assert w.rect_info()["num_shared_requests"] == 4


@pytest.mark.parametrize("lens,qsl,kw,status", [
    ([3, -1], [0, 1, 2], {}, kvq.E_INVALID_ARG), ([3, 4], [0, 2, 1], {}, kvq.E_INVALID_ARG),
    ([3, 4], [2, 3, 4], {}, kvq.E_INVALID_ARG), ([3, 4], [0, 1, 2], dict(hkv=3), kvq.E_UNSUPPORTED),
    ([3, 4], [0, 1, 2], dict(d=32), kvq.E_UNSUPPORTED)])
def test_cross_attention_refusals(lens, qsl, kw, status):
    with pytest.raises(kvq.KvqError) as e:
        kvq.get_cross_attention_metadata(2, 8, kw.get("hkv", 2), kw.get("d", 128), lens, qsl, "auto")
    assert e.value.status == status


def test_cross_attention_plans():
    """More queries than keys, encoders without keys, batches without queries."""
    s = kvq.get_cross_attention_metadata(3, 8, 2, 128, [3, 0, 7], [0, 900, 901, 901], "int8_per_token_head")
    assert s.rect_info()["num_units"] > 0 and s.info()["num_prefill_tiles"] == 0
    e = kvq.get_cross_attention_metadata(2, 8, 2, 128, [0, 0], [0, 0, 0], "int8_per_token_head")
    assert e.rect_info()["num_units"] == 0 and e.info()["num_kernel_launches"] == 0
    assert kvq.get_cross_attention_metadata(0, 8, 2, 128, [], [0], "auto").info()["num_kernel_launches"] == 0


def test_null_pointers():
    h, ws = ctypes.c_void_p(), ctypes.c_size_t()
    qsl = np.array([0, 1], np.int32)
    lens = np.array([9], np.int32)
    p = lambda a: ctypes.c_void_p(a.ctypes.data)  # noqa: E731
    f = kvq.lib.kvq_get_shared_prefix_metadata
    assert f(1, 8, 2, 128, p(lens), p(qsl), 1, None, p(lens), 0, 3, ctypes.byref(h), ctypes.byref(ws)) == kvq.E_INVALID_ARG
    assert f(1, 8, 2, 128, p(lens), p(qsl), 1, p(lens), None, 0, 3, ctypes.byref(h), ctypes.byref(ws)) == kvq.E_INVALID_ARG
    assert f(1, 8, 2, 128, p(lens), p(qsl), 0, None, p(lens), 0, 3, None, ctypes.byref(ws)) == kvq.E_INVALID_ARG
    assert kvq.lib.kvq_sched_get_rect_info(None, None) == kvq.E_INVALID_ARG
