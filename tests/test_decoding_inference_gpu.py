"""The decoding operators on tensors made in inference mode, which count no versions."""
from __future__ import annotations

import pytest
import torch

import mapreduce_prefix_scan_gb300 as ak

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("inside", [True, False])
def test_calls_in_place_on_inference_tensors(inside):
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    with torch.inference_mode():
        x, state, pool = torch.ones(2, 8, device="cuda"), torch.arange(12.0, device="cuda").reshape(2, 2, 3), torch.zeros(2, 8, device="cuda")
        gate, cache, logits = -torch.ones(2, 8, device="cuda"), torch.arange(6, device="cuda").reshape(3, 2), torch.eye(4, device="cuda")[None, :2]
        step = ak.ak_beam_select(logits, torch.zeros(1, 2, device="cuda"))
    with torch.inference_mode(inside):
        assert torch.equal(ak.ak_gated_recurrence_step(x, gate, pool), x) and torch.equal(pool, x)
        ak.ak_gated_recurrence(x, gate, out=x, state=pool[:1], state_out=pool[:1])
        torch.testing.assert_close(x[0], torch.full((8,), 1 + 0.36787944, device="cuda"))
        assert torch.equal(pool[0], x[1])
        ak.ak_beam_reorder(state, i32([[1, 1], [1, 0]]))
        assert state[:, :, 0].tolist() == [[3, 3], [9, 6]]
        ak.ak_blocks_copy(cache, i32([[0, 2]]))
        assert cache.tolist() == [[0, 1], [2, 3], [0, 1]]
        again = ak.ak_beam_select(logits, torch.zeros(1, 2, device="cuda"), out=step)
        assert again.tokens.tolist() == [[0, 1]] and again.parents.tolist() == [[0, 1]]
