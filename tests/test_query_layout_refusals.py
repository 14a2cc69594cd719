"""Queries and outputs that the attention calls cannot read or write as they lie:
the library takes no stride for them, so the binding refuses other layouts
before it hands their addresses over.  No call here reaches a kernel, so no GPU
is needed."""
import pytest
import torch

from int8_kv_cache_reshape_gb300 import kvq

T, HQ, H, D, DT = 5, 4, 2, 128, "int8_per_token_head"


def _bf(*n):
    return torch.zeros(n, dtype=torch.bfloat16)


def _common(**kw):
    i32 = lambda *n: torch.zeros(n, dtype=torch.int32)  # noqa: E731
    cache = torch.zeros((4, 16, H, kvq.cache_row_bytes(DT, D)), dtype=torch.uint8)
    a = dict(q=_bf(T, HQ, D), key_cache=cache, value_cache=cache, query_start_loc=i32(T + 1), seq_lens=i32(T),
             block_table=i32(T, 4), sm_scale=0.1, window=0, soft_cap=0.0, k_scale=1.0, v_scale=1.0, out=_bf(T, HQ, D),
             kv_cache_dtype=DT, heads_kv=H, stream=0)
    a.update(kw)
    return a


def _attention(fn, **kw):
    sched = kvq.get_scheduler_metadata(T, HQ, H, D, [9] * T, list(range(T + 1)), True, 0, DT)
    extra = {} if "static" in fn else dict(workspace=torch.zeros(256, dtype=torch.uint8))
    return getattr(kvq, fn)(sched, causal=True, **extra, **_common(**kw))


def _step(fn, **kw):
    io = {}
    if "io" in fn or "graph" in fn:
        io = dict(host_in=torch.zeros(64, dtype=torch.uint8), dev_in=torch.zeros(64, dtype=torch.uint8),
                  host_out=_bf(T, HQ, D), out_bytes=0)
    return getattr(kvq, fn)(key=_bf(T, H, D), value=_bf(T, H, D), slot_mapping=torch.zeros(T, dtype=torch.int64),
                            max_query_len=1, workspace=torch.zeros(256, dtype=torch.uint8), **io, **_common(**kw))


CALLS = [(_attention, "prepare_attention_with_kv_cache"), (_attention, "attention_with_kv_cache"),
         (_attention, "attention_with_kv_cache_static_scratch"), (_step, "prepare_decode_step"), (_step, "decode_step"),
         (_step, "prepare_decode_step_host_io"), (_step, "decode_step_graph")]
# queries as a fused projection and an in-place rotation leave them, every other
# head, transposed, of another type, without the heads' dimension
LAYOUTS = [_bf(T, HQ + 2 * H, D)[:, :HQ], _bf(T, 2 * HQ, D)[:, ::2], _bf(HQ, T, D).transpose(0, 1),
           _bf(T, HQ, 2 * D)[..., ::2], torch.zeros(T, HQ, D), torch.zeros((T, HQ, D), dtype=torch.float16)]


@pytest.mark.parametrize("name", ["q", "out"])
@pytest.mark.parametrize("layout", range(len(LAYOUTS)))
@pytest.mark.parametrize("call,fn", CALLS)
def test_layouts_that_are_refused(call, fn, name, layout):
    with pytest.raises(ValueError, match=f"^{name} must be"):
        call(fn, **{name: LAYOUTS[layout]})


def test_a_query_without_heads_is_refused():
    for call, fn in CALLS:
        with pytest.raises(ValueError):
            call(fn, q=_bf(T, HQ * D))


@pytest.mark.parametrize("call,fn", [c for c in CALLS if c[1].startswith("prepare")])
def test_layouts_that_are_taken(call, fn):
    """Rows side by side, some tokens of a longer batch, a single token (whose
    stride says nothing), an output longer than the batch."""
    call(fn)
    call(fn, q=_bf(9, HQ, D)[2:7], out=_bf(9, HQ, D)[:6])
    one = _bf(3, HQ + 2 * H, D)[:1, :HQ]
    p = call(fn, q=one, out=one)
    assert one.data_ptr() in [getattr(a, "value", a) for a in p.args]
    if "step" in fn:
        call(fn, out=None)
