"""What the binding refuses of gather_cache's and build_block_tables' tensors
before it hands their addresses to the library.  No call here reaches the
library's kernels: prepare_* only marshals arguments, so no GPU is needed."""
import pytest
import torch

from int8_kv_cache_reshape_gb300 import kvq


def _tables_tensors(R=3, width=4, **kw):
    i32 = lambda *n: torch.zeros(n, dtype=torch.int32)  # noqa: E731
    a = dict(query_start_loc=i32(R + 1), seq_lens=i32(R), free_blocks=i32(9), free_count=i32(1),
             block_table=i32(R, width), slot_mapping=torch.zeros(7, dtype=torch.int64), block_size=16, num_blocks=9,
             free_count_out=i32(1), status=i32(4), stream=0)
    a.update(kw)
    return a


def test_prepared_block_tables_take_the_width_of_the_view():
    assert kvq.prepare_build_block_tables(**_tables_tensors()).args[7].value == 4
    # rows of a taller table, and a view of some columns of one row
    wide = torch.zeros((5, 8), dtype=torch.int32)
    assert kvq.prepare_build_block_tables(**_tables_tensors(block_table=wide)).args[7].value == 8
    one = _tables_tensors(R=1, block_table=wide[2:3, :3])
    assert kvq.prepare_build_block_tables(**one).args[7].value == 3
    kvq.prepare_build_block_tables(**_tables_tensors(R=0, block_table=wide[:0]))


@pytest.mark.parametrize("name,make", [
    # some columns of a wider table: a request of more blocks would store past them
    ("block_table", lambda t: t.zeros((3, 8), dtype=t.int32)[:, :4]),
    ("block_table", lambda t: t.zeros((4, 3), dtype=t.int32).t()),
    ("block_table", lambda t: t.zeros((3, 8), dtype=t.int32)[:, ::2]),
    ("block_table", lambda t: t.zeros((3, 4), dtype=t.int64)),
    ("block_table", lambda t: t.zeros((2, 4), dtype=t.int32)),
    ("block_table", lambda t: t.zeros(12, dtype=t.int32)),
    ("query_start_loc", lambda t: t.zeros(4, dtype=t.int64)),
    ("query_start_loc", lambda t: t.zeros(5, dtype=t.int32)),
    ("query_start_loc", lambda t: t.zeros(8, dtype=t.int32)[::2]),
    ("seq_lens", lambda t: t.zeros(3, dtype=t.int64)),
    ("free_blocks", lambda t: t.zeros(18, dtype=t.int32)[::2]),
    ("free_blocks", lambda t: t.zeros(9, dtype=t.int64)),
    ("free_count", lambda t: t.zeros(0, dtype=t.int32)),
    ("free_count_out", lambda t: t.zeros(1, dtype=t.int64)),
    ("slot_mapping", lambda t: t.zeros(7, dtype=t.int32)),
    ("slot_mapping", lambda t: t.zeros(14, dtype=t.int64)[::2]),
    ("status", lambda t: t.zeros(3, dtype=t.int32)),
    ("status", lambda t: t.zeros(4, dtype=t.int64)),
])
def test_prepared_block_tables_refusals(name, make):
    with pytest.raises(ValueError):
        kvq.prepare_build_block_tables(**_tables_tensors(**{name: make(torch)}))


def _gather_tensors(H=3, D=128, T=5, dtype="int4_per_token_head", **kw):
    row = kvq.cache_row_bytes(dtype, D)
    a = dict(key_cache=torch.zeros((4, 16, H, row), dtype=torch.uint8),
             value_cache=torch.zeros((4, 16, H, row), dtype=torch.uint8),
             slot_mapping=torch.zeros(T, dtype=torch.int64), key_out=torch.zeros((T, H, D)),
             value_out=torch.zeros((T, H, D)), kv_cache_dtype=dtype, stream=0)
    a.update(kw)
    return a


@pytest.mark.parametrize("dtype", list(kvq.DTYPES))
def test_prepared_gather(dtype):
    for D in (64, 128, 256):
        kvq.prepare_gather_cache(**_gather_tensors(D=D, dtype=dtype))
    # views of wider rows, one head, no token
    buf = torch.zeros((5, 9, 128), dtype=torch.bfloat16)
    kvq.prepare_gather_cache(**_gather_tensors(dtype=dtype, key_out=buf[:, 1:4], value_out=buf[:, 5:8]))
    kvq.prepare_gather_cache(**_gather_tensors(H=1, dtype=dtype, key_out=buf[:, 1:2], value_out=buf[:, 5:6]))
    kvq.prepare_gather_cache(**_gather_tensors(T=0, dtype=dtype))


def test_prepared_gather_of_a_bf16_cache():
    cache = torch.zeros((4, 16, 3, 128), dtype=torch.bfloat16)
    kvq.prepare_gather_cache(**_gather_tensors(dtype="auto", key_cache=cache, value_cache=cache))


@pytest.mark.parametrize("kw", [
    # outputs of more heads (or another head_dim) than the cache: reads past it
    lambda: _gather_tensors(H=8, key_cache=_gather_tensors()["key_cache"], value_cache=_gather_tensors()["key_cache"]),
    lambda: _gather_tensors(value_cache=_gather_tensors(H=2)["value_cache"]),
    lambda: _gather_tensors(D=256, key_cache=_gather_tensors()["key_cache"],
                            value_cache=_gather_tensors()["key_cache"]),
    lambda: _gather_tensors(kv_cache_dtype="int8_per_token_head"),
    # fewer blocks of values than of keys
    lambda: _gather_tensors(value_cache=_gather_tensors()["value_cache"][:2]),
    lambda: _gather_tensors(key_cache=_gather_tensors()["key_cache"].float()),
    lambda: _gather_tensors(key_cache=_gather_tensors()["key_cache"].flatten(0, 1)),
    lambda: _gather_tensors(key_cache=torch.zeros((4, 16, 3, 160), dtype=torch.uint8)[..., :80]),
    lambda: _gather_tensors(key_cache=torch.zeros((8, 16, 3, 80), dtype=torch.uint8)[::2]),
    # heads or dims apart
    lambda: _gather_tensors(key_out=torch.zeros((5, 6, 128))[:, ::2]),
    lambda: _gather_tensors(value_out=torch.zeros((5, 3, 256))[..., ::2]),
    lambda: _gather_tensors(value_out=torch.zeros((5, 128, 3)).transpose(1, 2)),
    lambda: _gather_tensors(slot_mapping=torch.zeros(5, dtype=torch.int32)),
    lambda: _gather_tensors(slot_mapping=torch.zeros(10, dtype=torch.int64)[::2]),
    lambda: _gather_tensors(slot_mapping=torch.zeros((5, 2), dtype=torch.int64)),
    lambda: _gather_tensors(slot_mapping=torch.zeros(4, dtype=torch.int64)),
    lambda: _gather_tensors(key_out=torch.zeros((5, 3, 128), dtype=torch.float16)),
])
def test_prepared_gather_refusals(kw):
    with pytest.raises(ValueError):
        kvq.prepare_gather_cache(**kw())
