"""Orders in the decoding kernels' sources that a run need not show to be wrong."""
from __future__ import annotations

from test_sequence_sources import _kernel


def test_lanes_meet_before_they_read_one_anothers_candidates():
    """Each lane of a warp writes its candidate's total and token; the chosen ones are read by other lanes. With one
    beam the merge of the rows holds no barrier, so the warp needs one of its own."""
    body = _kernel("beam_search.cu", "k_beam_select")
    written = max(body.index("s.totals[k][lane] ="), body.index("s.tokens[k][lane] ="))
    merged = body.index("block_merge(list, s.picks")
    met = body.index("__syncwarp();", merged)
    read = min(body.index("s.totals[parent]"), body.index("s.tokens[parent]"))
    assert written < merged < met < read
    # every lane of the warp comes to it
    assert "if" not in body[merged:met]
