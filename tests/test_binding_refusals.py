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
