"""What the binding of the attention-layer operators refuses before any kernel
could see it.  Host only: tensors on the CPU, or metadata alone.
"""
import pytest
import torch

from gated_deltanet_prefill_gb300 import attn


def paged_metadata(table):
    """_check_paged on `table` as if it were on the GPU, with caches and lengths that fit."""
    n = table.shape[0]
    cache = (torch.Size((40, 16, 2, 64)), (2048, 128, 64, 1), torch.bfloat16, True)
    return attn._check_paged(cache, cache, (table.shape, table.stride(), table.dtype, True), (n, torch.int32, True),
                             (n + 1, torch.int32, True))


def test_block_table_rows_keep_their_stride():
    wide = torch.zeros(4, 15, dtype=torch.int32)
    n, _, _, stride, width, _ = paged_metadata(wide[:, :10])
    assert (n, stride, width) == (4, 15, 10)
    # a single row has no stride: any that is given goes
    for table in (wide[:1, :10], torch.zeros(10, dtype=torch.int32).expand(1, 10), wide.as_strided((1, 10), (3, 1))):
        assert paged_metadata(table)[0] == 1 and paged_metadata(table)[3] >= 10
    assert paged_metadata(wide[:, :0])[4] == 0 and paged_metadata(wide[:0])[0] == 0
    assert paged_metadata(wide[:, :1])[3:5] == (15, 1)


@pytest.mark.parametrize("shape,stride", [((4, 10), (0, 1)), ((4, 10), (5, 1)), ((2, 10), (9, 1)), ((4, 1), (0, 1)),
                                          ((4, 1), (0, 7))])
def test_block_table_rows_on_top_of_one_another_are_refused(shape, stride):
    """One row expanded to all sequences, rows that overlap: the kernels would read at strides that the table does not have."""
    table = torch.zeros(100, dtype=torch.int32).as_strided(shape, stride)
    with pytest.raises(ValueError, match="block_table"):
        paged_metadata(table)
