"""Block tables of the widest rows."""
from __future__ import annotations

import pytest
import torch

import mapreduce_prefix_scan_gb300 as ak

pytestmark = pytest.mark.gpu

WIDEST = (1 << 31) - 1


@pytest.mark.parametrize("width", [WIDEST, WIDEST - 127])
def test_rows_of_two_to_the_31_entries(width):
    """The pieces of a row are counted in 64 bits: its width and a piece's may pass 2^31 together."""
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    table = torch.full((1, width), -1, dtype=torch.int32, device="cuda")
    table[0, :5], table[0, -1] = i32([6, 1, 6, 7, 2]), 5
    lens = i32([5])
    refs = ak.ak_blocks_count(table, lens, block_size=1, blocks=9)
    assert refs.tolist() == [0, 1, 1, 0, 0, 0, 2, 1, 0]
    full = ak.ak_blocks_count(table, i32([WIDEST]), block_size=1, blocks=9)
    assert full.tolist() == [0, 1, 1, 0, 0, 1, 2, 1, 0]
    out, pairs, counts = ak.ak_blocks_compact(table, lens, refs, block_size=1, out=table)
    assert out is table and counts.tolist() == [2, 4] and pairs.tolist()[:3] == [[6, 0], [7, 3], [-1, -1]]
    assert table[0, :5].tolist() == [0, 1, 0, 3, 2] and int(table[0, -1]) == 5
    f = ak.ak_blocks_fork(table, i32([9]), i32([0, 0]), i32([8]), block_size=2, blocks=9)
    assert f.lens.tolist() == [9, 9] and f.counts.tolist() == [1] and f.pairs.tolist() == [[2, 8], [-1, -1]]
    assert f.table[:, :5].tolist() == [[0, 1, 0, 3, 2], [0, 1, 0, 3, 8]]
    assert (f.table[:, 5:] == -1).all()
