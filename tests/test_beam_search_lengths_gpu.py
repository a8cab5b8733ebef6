"""Beam selection with lengths that no beam has."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import decoding_reference as ref
import mapreduce_prefix_scan_gb300 as ak

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("ended", [False, True])
@pytest.mark.parametrize("penalty", [0.0, 0.6, 1.0, 2.0, 3.0, -1.0])
def test_a_negative_power_of_a_length_ranks_nothing(penalty, ended):
    """A rank over a number below 0 would turn the order of a beam's candidates round: such a beam has none, and the
    others keep theirs."""
    n, k, v = 3, 5, 900
    g = torch.Generator().manual_seed(7)
    logits, scores = torch.randn(n, k, v, generator=g) * 2.5, -torch.rand(n, k, generator=g) * 4
    lengths = torch.tensor([-3, 4, -2147483648, 9, -2], dtype=torch.int32).repeat(n, 1)
    done = torch.zeros(n, k, dtype=torch.bool)
    done[:, 0] = ended
    r = ak.ak_beam_select(logits.cuda(), scores.cuda(), done=done.cuda(), lengths=lengths.cuda(), end_token=3, length_penalty=penalty)
    taken = lengths.numpy().astype(np.float64) + ~done.numpy()
    with np.errstate(all="ignore"):
        none = np.zeros((n, k), bool) if penalty == 0 else ~(taken**penalty >= 0)
    s, t, p, d, m = ref.beam_step(logits.numpy(), np.where(none, -np.inf, scores.numpy()), done.numpy(), lengths.numpy(), 3, penalty)
    assert r.tokens.tolist() == t.tolist() and r.parents.tolist() == p.tolist()
    assert r.done.tolist() == d.tolist() and r.lengths.tolist() == m.tolist()
