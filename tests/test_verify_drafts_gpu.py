"""ak_verify_drafts against the definition in 64 bits. Whole numbers: exact.
The inputs make near-ties of float32 scores (relative 2^-23) that 64 bits
would order otherwise too rare to meet (a few hundred rows of random noise);
exact ties are planted and go to the lowest index."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import mapreduce_prefix_scan_gb300 as ak
from sequence_reference import verify

pytestmark = pytest.mark.gpu


def _softmax(x):
    e = np.exp(x - x.max(-1, keepdims=True))
    return (e / e.sum(-1, keepdims=True)).astype(np.float32)


def _case(seed, n, k, vocab, near=0.6):
    rng = np.random.default_rng(seed)
    x = rng.normal(0, 2, (n, k + 1, vocab))
    p, q = _softmax(x), _softmax(x[:, :k] + rng.normal(0, near, (n, k, vocab)))
    drafts = np.array([[rng.choice(vocab, p=q[r, j].astype(np.float64) / q[r, j].astype(np.float64).sum())
                        for j in range(k)] for r in range(n)]).reshape(n, k)
    return p, q, drafts, rng.random((n, k), dtype=np.float32), rng.exponential(1, (n, vocab)).astype(np.float32) + 1e-12


def _run(p, q, drafts, counts, u, noise, dtype=torch.float32, **kw):
    c = lambda x, t: None if x is None else torch.tensor(np.ascontiguousarray(x), device="cuda").to(t)
    tokens, accepted = ak.ak_verify_drafts(c(p, dtype), c(drafts, torch.int32), c(u, torch.float32),
                                           c(noise, torch.float32), draft_probs=c(q, dtype),
                                           draft_counts=c(counts, torch.int32), **kw)
    return tokens.cpu().numpy(), accepted.cpu().numpy()


def _same(got, want):
    assert np.array_equal(got[1], want[1]), "accepted"
    assert np.array_equal(got[0], want[0]), "tokens"


@pytest.mark.parametrize("n,k,vocab", [(1, 1, 1), (1, 3, 5), (3, 4, 1000), (2, 2, 32003), (1, 1, 40000), (30, 5, 513),
                                       (70, 40, 130), (400, 1, 2049), (5, 0, 777), (2, 3, 65536)])
@pytest.mark.parametrize("drafted", [True, False])
def test_against_definition(n, k, vocab, drafted):
    p, q, d, u, e = _case(n + vocab, n, k, vocab)
    _same(_run(p, q if drafted else None, d, None, u, e), verify(p, q if drafted else None, d, None, u, e))


@pytest.mark.parametrize("drafted", [True, False])
@pytest.mark.parametrize("vocab", [1000, 8191])
def test_bf16_and_counts(drafted, vocab):
    p, q, d, u, e = _case(3, 40, 3, vocab)
    r = lambda x: torch.tensor(x).bfloat16().float().numpy()
    p, q = r(p), r(q)
    counts = np.array([0, 1, 2, 3, -4, 9] * 7)[:40]
    q_ = q if drafted else None
    _same(_run(p, q_, d, counts, u, e, dtype=torch.bfloat16), verify(p, q_, d, counts, u, e))


def test_same_distributions_keep_everything_and_leave_p_to_decide():
    p, q, d, u, e = _case(4, 6, 3, 900)
    q = p[:, :3].copy()
    d = np.argmax(q, -1)
    t, a = _run(p, q, d, None, u, e)
    assert (a == 3).all()
    _same((t, a), verify(p, q, d, None, u, e))
    # a draft of probability zero under an equal distribution is refused, and nothing is left over: p decides
    p[:, :, 7] = 0
    q = p[:, :3].copy()
    d[:] = 7
    got = _run(p, q, d, None, u, e)
    assert (got[1] == 0).all()
    _same(got, verify(p, q, d, None, u, e))


def test_ties_go_to_the_lowest_index_and_bounds_of_u():
    n, k, vocab = 4, 2, 20000
    p = np.full((n, k + 1, vocab), 1 / vocab, np.float32)
    q = np.zeros((n, k, vocab), np.float32)
    q[:, :, 3] = 1
    d = np.full((n, k), 3)
    e = np.full((n, vocab), 0.5, np.float32)
    e[1, 500:] = 0.25
    u = np.full((n, k), 0.75, np.float32)
    u[3] = 0.0  # zero keeps any draft that the target allows
    want = verify(p, q, d, None, u, e)
    got = _run(p, q, d, None, u, e)
    _same(got, want)
    assert got[0][0, 0] == 0 and got[0][1, 0] == 500 and got[1][3] == k


def test_draft_tokens_outside_the_vocabulary_nan_and_empty_rows():
    p, q, d, u, e = _case(9, 8, 2, 300)
    d[0, 0], d[1, 1], d[2, 0] = -1, 300, 2**30
    p[3] = 0                      # nothing to draw from
    p[4, :, 5] = np.nan           # passed over
    p[5, 0] = np.nan
    e[6, 10] = np.nan
    e[7, 11] = 0                  # an infinite score wins
    _same(_run(p, q, d, None, u, e), verify(p, q, d, None, u, e))
    _same(_run(p, None, d, None, u, e), verify(p, None, d, None, u, e))


def test_strided_rows():
    p, q, d, u, e = _case(10, 5, 3, 700)
    pad = lambda x: torch.nn.functional.pad(torch.tensor(x, device="cuda"), (3, 2))
    P, Q, E = pad(p)[..., 3:703], pad(q)[..., 3:703], pad(e)[..., 3:703]
    t, a = ak.ak_verify_drafts(P, torch.tensor(d, device="cuda").int(), torch.tensor(u, device="cuda"), E, draft_probs=Q)
    _same((t.cpu().numpy(), a.cpu().numpy()), verify(p, q, d, None, u, e))


def test_emitted_tokens_follow_the_target():
    """One draft, 40000 requests of one small distribution: the first emitted token is distributed as p.
    Tolerance: five standard deviations of a count."""
    n, vocab = 40000, 11
    rng = np.random.default_rng(12)
    p1, q1 = _softmax(rng.normal(0, 1, vocab)), _softmax(rng.normal(0, 1, vocab))
    p, q = np.broadcast_to(p1, (n, 2, vocab)), np.broadcast_to(q1, (n, 1, vocab))
    d = rng.choice(vocab, (n, 1), p=q1.astype(np.float64) / q1.astype(np.float64).sum())
    t, _ = _run(p, q, d, None, rng.random((n, 1), dtype=np.float32), rng.exponential(1, (n, vocab)).astype(np.float32) + 1e-12)
    seen = np.bincount(t[:, 0], minlength=vocab)
    assert (np.abs(seen - n * p1) <= 5 * np.sqrt(n * p1 * (1 - p1)) + 1).all()


def test_rows_beyond_2_31_values():
    n, k, vocab = 3000, 5, 128000
    p = torch.zeros(n, k + 1, vocab, device="cuda")
    ps, qs, d, u, e = _case(15, 2, k, vocab)
    p[-2:] = torch.tensor(ps, device="cuda")
    drafts = torch.full((n, k), -1, dtype=torch.int32, device="cuda")
    drafts[-2:] = torch.tensor(d, device="cuda").int()
    uniform = torch.zeros(n, k, device="cuda")
    uniform[-2:] = torch.tensor(u, device="cuda")
    noise = torch.ones(n, vocab, device="cuda")
    noise[-2:] = torch.tensor(e, device="cuda")
    t, a = ak.ak_verify_drafts(p, drafts, uniform, noise)
    _same((t[-2:].cpu().numpy(), a[-2:].cpu().numpy()), verify(ps, None, d, None, u, e))
    assert (a[:-2] == 0).all() and (t[:-2] == -1).all()
