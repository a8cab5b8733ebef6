"""How far the logarithm of a row's sum of exponentials is off."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import mapreduce_prefix_scan_gb300 as ak

pytestmark = pytest.mark.gpu

ROWS = {
    "ordinary": lambda x, at: x * 2.5,
    "sharp": lambda x, at: x * 6,
    "flat": lambda x, at: x * 0.3,
    "all but one far below": lambda x, at: torch.where(at == 5, torch.tensor(18.0), x * 2.5),
    "rising": lambda x, at: at / at.numel() * 20 + x * 0.01,
}


@pytest.mark.parametrize("v", [5003, 32003, 128000])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("name", ROWS)
def test_a_logarithm_of_a_sum_of_exponentials(name, dtype, v):
    """A score that cancels the logarithm leaves what it is off by.

    An exponential is off by 2^-22 (its instruction) and by its argument: a subtraction's and a product's half steps and
    log2 e as a float32 (1.3e-8 of it), in all d (2^-23 + 1.3e-8) < d 2^-22.8 for a logit d below the largest that its
    thread has met, and as much again for what that one lies below the row's. Sums of at most eight: four half steps,
    2^-22. A thread that meets a larger logit scales its sum: 2 ulp and a half step, less than 2^-21.6; so do the block's
    and the slices' joins, twice at most. Sums of sums are compensated. The result is a difference of 64-bit numbers rounded to
    float32, next to 0."""
    n = 700  # requests of one beam: rows whole, the 64 different ones over and over
    g = torch.Generator().manual_seed(v)
    x = ROWS[name](torch.randn(64, v, generator=g), torch.arange(v).float()).to(dtype)
    d = x.double()
    top = d.amax(-1)
    p = torch.exp(d - top[:, None])
    lse = p.sum(-1).log()
    below = ((top[:, None] - d) * p).sum(-1) / p.sum(-1)
    # larger logits that a thread meets, at most: of each 256 groups of 16 bytes one is its own
    group = 16 // dtype.itemsize
    per = -(-v // (group * 256))
    own = torch.full((64, per * 256 * group), -float("inf"), dtype=torch.float64)
    own[:, :v] = d
    best = own.reshape(64, per, 256, group).amax(-1).cummax(1).values
    met = (best[:, 1:] > best[:, :-1]).sum(1).amax(-1)
    bound = 2.0**-21 + below * 2.0**-22.8 + (met + 2) * 2.0**-21.6
    score = lse.float()
    pick = torch.arange(n) % 64
    r = ak.ak_beam_select(x.cuda()[pick.cuda()][:, None], score[pick].cuda()[:, None])
    off = (r.scores[:, 0].double().cpu() - (score.double() - lse)[pick]).abs()
    # what is left is of the order of the bound, and rounded to float32
    assert (off <= (bound * (1 + 2.0**-20))[pick]).all(), float((off / bound[pick]).max())
    assert np.isfinite(float(off.max()))
