"""ak_verify_drafts where u * q(d) and p(d) differ by less than a float32 rounding: the product is compared exactly."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import mapreduce_prefix_scan_gb300 as ak

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("smallest", [2.0**-10, 2.0**-148])  # (probabilities down to the smallest float32 values)
def test_a_product_that_rounds_to_the_target(smallest):
    n, vocab = 4000, 5
    rng = np.random.default_rng(1)
    u = rng.random(n, dtype=np.float32)
    q = (rng.random(n) * (1 - smallest) + smallest).astype(np.float32)
    if smallest < 2.0**-126:
        q = (rng.integers(1, 1 << 20, n) * smallest).astype(np.float32)
    p = (u * q).astype(np.float32)  # rounded: above, below or at the product
    exact = u.astype(np.float64) * q.astype(np.float64)
    want = exact < p.astype(np.float64)
    assert 0.2 * n < want.sum() < 0.8 * n
    P, Q = np.full((n, 2, vocab), 0.25, np.float32), np.full((n, 1, vocab), 0.25, np.float32)
    P[:, 0, 3], Q[:, 0, 3] = p, q
    dev = lambda x, t=torch.float32: torch.tensor(x, device="cuda").to(t)
    _, accepted = ak.ak_verify_drafts(dev(P), dev(np.full((n, 1), 3), torch.int32), dev(u[:, None]),
                                      torch.ones(n, vocab, device="cuda"), draft_probs=dev(Q))
    assert np.array_equal(accepted.cpu().numpy(), want.astype(np.int64))
