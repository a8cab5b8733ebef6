"""Beam selection where a row's best logits lie in few threads' columns, next to one another."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import decoding_reference as ref
import mapreduce_prefix_scan_gb300 as ak

pytestmark = pytest.mark.gpu

THREADS = 256


def _check(logits, scores, requests, keep):
    """Every one of `requests` equal requests against the definition, twice with equal bits."""
    call = lambda: ak.ak_beam_select(logits.expand(requests, -1, -1), scores.expand(requests, -1).contiguous(), keep=keep)  # noqa: E731
    r, again = call(), call()
    assert all(torch.equal(a, b) for a, b in zip(r, again))
    s, t, p, _, _ = ref.beam_step(logits.float().cpu().numpy(), scores.cpu().numpy(), keep=keep)
    assert (r.tokens.cpu().numpy() == t).all() and (r.parents.cpu().numpy() == p).all()
    # the half step of the result, and the exponentials' 2^-20 in their sum's logarithm
    assert (np.abs(r.scores.double().cpu().numpy() - s) <= 2.0**-24 * np.abs(s) + 2.0**-20).all()


def _crowded(k, v, dtype, held, seed, rest):
    """Logits whose largest lie in the columns that `held` threads of a block read, if it takes rows whole."""
    g = torch.Generator().manual_seed(seed)
    group = 16 // dtype.itemsize
    high = torch.arange(v) // group % THREADS < held
    x = torch.randn(1, k, v, generator=g)
    x = torch.where(high, x + 20, x if rest else torch.tensor(-float("inf"))).to(dtype)
    return x, int(high.sum())


# (beams, kept, requests): rows in two slices, rows whole, rows whole for many requests, one beam
@pytest.mark.parametrize("k,keep,requests", [(8, 8, 1), (16, 16, 1), (8, 8, 45), (1, 32, 700)])
@pytest.mark.parametrize("v,held", [(32000, 7), (32000, 31), (32768, 15), (50257, 6), (50257, 12), (128000, 3), (128000, 7), (152064, 2),
                                    (262144, 1), (262144, 5)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_thousands_of_candidates_in_few_threads(dtype, v, held, k, keep, requests):
    """Fewer threads than are kept hold all that is large, so that no bound keeps any of it out."""
    if held >= keep:
        held = keep - 1
    logits, high = _crowded(k, v, dtype, held, v + held + k, rest=True)
    assert high > 800
    scores = -torch.rand(1, k, generator=torch.Generator().manual_seed(v))
    _check(logits.cuda(), scores.cuda(), requests, keep)


@pytest.mark.parametrize("k,keep,requests", [(8, 8, 1), (16, 32, 1), (8, 8, 45)])
@pytest.mark.parametrize("v,held", [(32768, 15), (128000, 7), (128000, 1), (200001, 256)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_all_other_tokens_banned(dtype, v, held, k, keep, requests):
    logits, _ = _crowded(k, v, dtype, held, v + held, rest=False)
    _check(logits.cuda(), torch.zeros(1, k).cuda(), requests, keep)


@pytest.mark.parametrize("v", [2048, 8192, 128000])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_equal_logits_everywhere(dtype, v):
    """Every column a candidate until the bound tells columns apart."""
    for k, keep, requests in ((8, 32, 1), (16, 16, 2), (2, 2, 400)):
        _check(torch.ones(1, k, v).to(dtype).cuda(), torch.zeros(1, k).cuda(), requests, keep)
