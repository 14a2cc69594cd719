"""The 4-bit cache dtype on the host: its name, row size and plan sizes; the
oracle's 4-bit rows pinned by the format's definition; refusals of
gather_cache and build_block_tables (argument checks come before any device
call, so no GPU is needed)."""
import ctypes

import numpy as np
import pytest

import oracle
from int8_kv_cache_reshape_gb300 import kvq

DT = kvq.DTYPES["int4_per_token_head"]


def test_name_and_row_bytes():
    assert kvq.parse_kv_cache_dtype("int4_per_token_head") == DT == 6
    for D in (64, 128, 192, 256):
        assert kvq.cache_row_bytes("int4_per_token_head", D) == D // 2 + 16
        assert oracle.row_bytes(oracle.INT4_PER_TOKEN_HEAD, D) == D // 2 + 16
    for D in (16, 32, 48, 96, 0, -64):
        with pytest.raises(kvq.KvqError):
            kvq.cache_row_bytes("int4_per_token_head", D)


def test_plan_sizes_follow_the_row():
    sl, ql = np.array([300], np.int32), np.array([0, 1], np.int32)
    info = kvq.get_scheduler_metadata(1, 32, 8, 128, sl, ql, True, 0, "int4_per_token_head").info()
    assert info["row_bytes"] == 80 and info["decode_chunk_bytes"] == 2 * 32 * 80


def _bits(x):
    """bf16 patterns of float32 values that are bf16 numbers."""
    return (np.asarray(x, np.float32).view(np.uint32) >> 16).astype(np.uint16)


def _bf16(x):
    """float32 values rounded to bf16 by truncation (any bf16 will do)."""
    return (np.asarray(x, np.float32).view(np.uint32) & 0xFFFF0000).view(np.float32)


def _write(x):
    T, D = x.shape
    kc = np.zeros((T, 1, 1, D // 2 + 16), np.uint8)
    vc = kc.copy()
    b = _bits(x).reshape(T, 1, D)
    oracle.reshape_and_cache(b, b, kc, vc, np.arange(T), oracle.INT4_PER_TOKEN_HEAD, 1.0, 1.0, 1)
    assert np.array_equal(kc, vc)
    return kc.reshape(T, -1)


def _codes(rows, D):
    """Codes by the header's words: nibble j of word w is dim 8 w + 2 j (j <
    4) or 8 w + 2 (j - 4) + 1."""
    words = np.ascontiguousarray(rows[:, : D // 2]).view("<u4")
    out = np.zeros((rows.shape[0], D), np.int32)
    for w in range(D // 8):
        for j in range(8):
            out[:, 8 * w + (2 * j if j < 4 else 2 * (j - 4) + 1)] = (words[:, w] >> (4 * j) & 15).astype(np.int32) - 8
    return out


@pytest.mark.parametrize("D", [64, 128, 256])
def test_oracle_rows_follow_the_definition(D):
    rng = np.random.default_rng(D)
    x = _bf16(rng.standard_normal((200, D)) * np.exp(3 * rng.standard_normal((200, 1))))
    x[0] = 0                      # a zero row
    x[1, : D // 8] = 0            # a zero group
    x[2] = 1.0e-39                # subnormals
    x[3] = _bf16([3.0e38])[0]     # near the largest
    x[4] = 7.0                    # quotients next to .5
    x[4, :6] = [0.5, 1.5, 2.5, -3.5, -0.5, 6.5]
    x[5, 1:] = 0                  # one element
    x = _bf16(x)
    rows = _write(x)
    f = np.float32
    amax = np.abs(x).max(1)
    s = (amax / f(889)).astype(f)
    assert np.array_equal(rows[:, D // 2: D // 2 + 4].copy().view("<f4")[:, 0], s)
    assert not rows[:, D // 2 + 12:].any()
    code = _codes(rows, D)
    g = x.reshape(200, 8, D // 8)
    with np.errstate(invalid="ignore", divide="ignore"):
        m = np.ceil(((np.abs(g).max(2) / s[:, None]).astype(f) / f(7)).astype(f))
        m = np.where(s[:, None] > 0, np.minimum(m, 127), 0)
        step = (s[:, None] * m.astype(f)).astype(f)
        want = np.clip(np.rint((g / step[:, :, None]).astype(f)), -7, 7)
    want = np.where(step[:, :, None] > 0, want, 0)
    assert np.array_equal(rows[:, D // 2 + 4: D // 2 + 12], m.astype(np.uint8))
    assert np.array_equal(code.reshape(200, 8, -1), want.astype(np.int32))
    # a value is off by at most half its group's step (normal rows: the step's
    # own rounding adds less than 2^-20 of it)
    val = code.reshape(200, 8, -1).astype(np.float64) * step[:, :, None]
    err = np.abs(val - g)
    assert (err[6:] <= step[6:, :, None] * (0.5 + 2.0 ** -20)).all()


def test_oracle_attention_reads_4bit_rows():
    """One key: the output is the row's value."""
    D = 64
    rng = np.random.default_rng(9)
    x = _bf16(rng.standard_normal((1, D)))
    rows = _write(x).reshape(1, 1, 1, -1)
    q = _bits(_bf16(rng.standard_normal((1, D)))).reshape(1, 1, D)
    out = oracle.attention(q, rows, rows, [0, 1], [1], [[0]], 1, 1, oracle.INT4_PER_TOKEN_HEAD, 0.1, True, 0, 0.0,
                           1.0, 1.0)
    tail = rows[0, 0, 0, D // 2:]
    s = tail[:4].copy().view("<f4")[0]
    m = np.repeat(tail[4:12].astype(np.float64), D // 8)
    assert np.allclose(out[0, 0], _codes(rows.reshape(1, -1), D)[0] * m * s, rtol=2.0 ** -23, atol=0)


# ---- refusals ------------------------------------------------------------------

P = ctypes.c_void_p(256)


def _gather_args(**kw):
    a = dict(kc=P, vc=P, nb=4, bs=16, h=2, D=128, dt=DT, ks=1.0, vs=1.0, slots=P, T=3, fp32=1, ko=P, vo=P,
             kst=256, vst=256)
    a.update(kw)
    return list(a.values()) + [None]


@pytest.mark.parametrize("kw,want", [
    (dict(dt=7), kvq.E_INVALID_ARG), (dict(dt=-1), kvq.E_INVALID_ARG), (dict(D=96), kvq.E_UNSUPPORTED),
    (dict(T=-1), kvq.E_INVALID_ARG), (dict(h=0), kvq.E_INVALID_ARG), (dict(bs=0), kvq.E_INVALID_ARG),
    (dict(nb=-1), kvq.E_INVALID_ARG), (dict(fp32=2), kvq.E_INVALID_ARG), (dict(kc=None), kvq.E_INVALID_ARG),
    (dict(vc=None), kvq.E_INVALID_ARG), (dict(slots=None), kvq.E_INVALID_ARG), (dict(ko=None), kvq.E_INVALID_ARG),
    (dict(vo=None), kvq.E_INVALID_ARG), (dict(kst=248), kvq.E_INVALID_ARG), (dict(vst=260), kvq.E_INVALID_ARG),
    (dict(ko=ctypes.c_void_p(264)), kvq.E_INVALID_ARG), (dict(slots=ctypes.c_void_p(260)), kvq.E_INVALID_ARG),
    (dict(dt=1, ks=float("nan")), kvq.E_INVALID_ARG), (dict(T=0, kc=None, ko=None), kvq.OK),
])
def test_gather_refusals(kw, want):
    assert kvq.lib.kvq_gather_cache(*_gather_args(**kw)) == want


def _table_args(**kw):
    a = dict(R=2, qsl=P, sl=P, free=P, cap=4, count=P, table=P, width=3, slots=P, T=5, bs=16, nb=4, out=P, status=P)
    a.update(kw)
    return list(a.values()) + [None]


@pytest.mark.parametrize("kw,want", [
    (dict(R=-1), kvq.E_INVALID_ARG), (dict(T=-1), kvq.E_INVALID_ARG), (dict(cap=-1), kvq.E_INVALID_ARG),
    (dict(bs=0), kvq.E_INVALID_ARG), (dict(nb=-1), kvq.E_INVALID_ARG), (dict(width=0), kvq.E_INVALID_ARG),
    (dict(T=1 << 31), kvq.E_UNSUPPORTED), (dict(cap=1 << 31), kvq.E_UNSUPPORTED),
    (dict(count=None), kvq.E_INVALID_ARG), (dict(out=None), kvq.E_INVALID_ARG), (dict(status=None), kvq.E_INVALID_ARG),
    (dict(free=None), kvq.E_INVALID_ARG), (dict(qsl=None), kvq.E_INVALID_ARG), (dict(sl=None), kvq.E_INVALID_ARG),
    (dict(table=None), kvq.E_INVALID_ARG), (dict(slots=None), kvq.E_INVALID_ARG),
    (dict(slots=ctypes.c_void_p(260)), kvq.E_INVALID_ARG), (dict(qsl=ctypes.c_void_p(258)), kvq.E_INVALID_ARG),
])
def test_block_table_refusals(kw, want):
    assert kvq.lib.kvq_build_block_tables(*_table_args(**kw)) == want


def test_attention_refuses_a_schedule_of_another_width():
    """4-bit caches run only with a schedule planned for them."""
    sl, ql = np.array([64], np.int32), np.array([0, 1], np.int32)
    s = kvq.get_scheduler_metadata(1, 8, 2, 128, sl, ql, True, 0, "int8_per_token_head")
    rc = kvq.lib.kvq_attention_with_kv_cache(s.handle, 8, 2, 128, DT, *([P] * 6), 4, 16, 8, 0.1, 1, 0, 0.0, None, None,
                                             1.0, 1.0, P, None, 0, None)
    assert rc == kvq.E_SCHED_MISMATCH
