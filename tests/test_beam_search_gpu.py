"""Beam search's step and the reordering of states against the definition in 64 bits."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import decoding_reference as ref
import mapreduce_prefix_scan_gb300 as ak

pytestmark = pytest.mark.gpu


def _check(logits, scores, done=None, lengths=None, end=-1, penalty=0.0, keep=None, **kw):
    r = ak.ak_beam_select(logits, scores, done=done, lengths=lengths, end_token=end, length_penalty=penalty, keep=keep, **kw)
    np_ = lambda t: None if t is None else (t.float() if t.is_floating_point() else t).cpu().numpy()  # noqa: E731
    s, t, p, d, m = ref.beam_step(np_(logits), np_(scores), np_(done), np_(lengths), end, penalty, keep)
    assert r.tokens.tolist() == t.tolist() and r.parents.tolist() == p.tolist()
    assert r.done.tolist() == d.tolist() and r.lengths.tolist() == m.tolist()
    got = r.scores.double().cpu().numpy()
    fine = np.isfinite(s)
    assert (fine == np.isfinite(got)).all() and (got[~fine] == -np.inf).all()
    got, s = got[fine], s[fine]
    # the stored float32's half step; exponentials off by 2^-21 in all (2 ulp of ex2 and its rounded argument, below 8 where
    # a term still weighs) give a logarithm off by as much
    assert (np.abs(got - s) <= 2.0**-24 * np.abs(s) + 2.0**-20).all()
    return r


def _random(n, k, v, dtype, seed=0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(n, k, v, generator=g) * 2.5).to(dtype).cuda(), (-torch.rand(n, k, generator=g) * 4).cuda()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n,k,v", [(1, 1, 1), (1, 4, 3), (3, 2, 1000), (2, 5, 1001), (1, 4, 32003), (7, 8, 4097), (2, 16, 5003),
                                   (1, 32, 2500), (2, 31, 40), (170, 3, 259), (1, 1, 200001), (700, 2, 65)])
def test_select(n, k, v, dtype):
    logits, scores = _random(n, k, v, dtype, n + k + v)
    _check(logits, scores)


@pytest.mark.parametrize("penalty", [0.0, 0.6, 1.0, -0.5])
def test_ended_beams_and_lengths(penalty):
    n, k, v = 12, 6, 300
    logits, scores = _random(n, k, v, torch.float32, 5)
    g = torch.Generator().manual_seed(1)
    done = (torch.rand(n, k, generator=g) < 0.4).cuda()
    done[3] = True
    logits[done] = float("nan")  # not read
    lengths = torch.randint(1, 30, (n, k), generator=g, dtype=torch.int32).cuda()
    for end in (2, v - 1, -1):
        _check(logits, scores, done, lengths, end, penalty)
    _check(logits, scores, done, None, 0, 0.0)


@pytest.mark.parametrize("k,keep", [(1, 8), (4, 1), (5, 32), (32, 3)])
def test_another_number_of_beams(k, keep):
    logits, scores = _random(4, k, 700, torch.bfloat16, keep)
    _check(logits, scores, keep=keep)


def test_ties_go_to_the_lowest_beam_and_token():
    # one value everywhere, at sizes on either side of a round of loads and of a slice
    for v in (5, 31, 1024, 1027, 8200):
        for n in (1, 300):
            logits = torch.zeros(n, 4, v, device="cuda")
            r = _check(logits, torch.full((n, 4), -1.0, device="cuda"))
            assert r.parents[0].tolist() == ([0] * 4) and r.tokens[0].tolist() == [0, 1, 2, 3]
    # equal rows at four alignments: the same candidates tie, the lower beam first
    for dtype in (torch.float32, torch.bfloat16):
        row = (torch.randn(1, 1, 20003) * 3).to(dtype).cuda()
        r = _check(row.expand(2, 6, 20003).contiguous(), torch.zeros(2, 6, device="cuda"))
        assert r.parents[0].tolist() == [0, 1, 2, 3, 4, 5]
        _check(row.expand(2, 6, 20003), torch.zeros(2, 6, device="cuda"))  # (by stride 0)
    # zeros of both signs are one value
    logits = torch.full((1, 2, 600), -5.0, device="cuda")
    logits[0, 0, 500], logits[0, 0, 77], logits[0, 0, 300] = 0.0, -0.0, 0.0
    r = _check(logits, torch.tensor([[0.0, -3.0]], device="cuda"))
    assert r.tokens.tolist() == [[77, 300]]
    # few distinct values: ties among thousands
    logits = torch.randint(0, 3, (3, 8, 9001), device="cuda").bfloat16()
    _check(logits, torch.zeros(3, 8, device="cuda"))


def test_candidates_that_one_thread_holds():
    """The best of a row a round of loads apart, so that one thread sees them all."""
    for v, k in ((128000, 8), (50000, 32)):
        logits = torch.randn(1, k, v, device="cuda")
        at = torch.arange(0, v, 1024, device="cuda")
        for j in range(0, k, 3):
            logits[0, j, at] = 20 + torch.rand(at.numel(), device="cuda")
        _check(logits, torch.zeros(1, k, device="cuda"))
        if k == 8:  # rows whole
            _check(logits.expand(45, k, v), torch.zeros(45, k, device="cuda"))


def test_banned_tokens_and_lost_rows():
    inf, nan = float("inf"), float("nan")
    logits, scores = _random(1, 5, 900, torch.float32, 9)
    logits[0, 0, 3:] = -inf             # three left
    logits[0, 1] = -inf                 # none
    logits[0, 2, 17] = nan              # no row
    logits[0, 3, 899] = inf             # no row
    scores[0, 4] = -inf                 # no beam
    r = _check(logits, scores)
    assert (r.parents[0, :3] == 0).all() and (r.parents[0, 3:] == -1).all() and (r.scores[0, 3:] == -inf).all()
    for bad in (nan, inf, -inf):
        scores[0, 0] = bad
        r = _check(logits, scores)
        assert (r.tokens == -1).all() and (r.parents == -1).all() and r.done.all() and not r.lengths.any()
    # the type's lowest value is a value
    logits = torch.full((1, 2, 40), torch.finfo(torch.float32).min, device="cuda")
    logits[0, 1, 20] = 0.0
    _check(logits, torch.zeros(1, 2, device="cuda"))
    # large logits: their differences count
    logits = torch.full((1, 3, 50), 3e38, device="cuda")
    logits[0, :, 7] = 3.1e38
    _check(logits, torch.tensor([[-1.0, -2.0, -0.5]], device="cuda"))


def test_views():
    """Rows at strides of their own; outputs into an earlier step's tensors."""
    wide = torch.randn(3, 4, 2, 1100, device="cuda")
    logits = wide[:, :, 1, 1: 1051]
    scores = torch.randn(3, 4, device="cuda")
    a = _check(logits, scores)
    b = ak.ak_beam_select(logits.contiguous(), scores, out=a)
    assert b.tokens.data_ptr() == a.tokens.data_ptr()


def test_a_step_in_its_own_tensors():
    """An earlier step's tensors are inputs and outputs at once."""
    n, k, v = 40, 5, 700
    logits, scores = _random(n, k, v, torch.float32, 3)
    a = ak.ak_beam_select(logits, scores, end_token=7, length_penalty=0.7)
    for seed in range(3):
        logits = _random(n, k, v, torch.float32, 50 + seed)[0]
        logits[:, :, 7] += 6
        want = ak.ak_beam_select(logits, a.scores, done=a.done, lengths=a.lengths, end_token=7, length_penalty=0.7)
        b = ak.ak_beam_select(logits, a.scores, done=a.done, lengths=a.lengths, end_token=7, length_penalty=0.7, out=a)
        assert b.scores.data_ptr() == a.scores.data_ptr() and all(torch.equal(x, y) for x, y in zip(b, want))
    assert a.done.any() and not a.done.all()


def test_ranks_that_tie_after_the_division():
    """-49 over 49 tokens and -50 over 50 are one rank: the lowest beam. Reciprocals would tell them apart."""
    m = torch.tensor([[50, 49, 7]], dtype=torch.int32, device="cuda")
    r = ak.ak_beam_select(torch.zeros(1, 3, 9, device="cuda"), -m.float(), done=torch.ones(1, 3, dtype=torch.bool, device="cuda"),
                          lengths=m, end_token=1, length_penalty=1.0)
    assert r.parents.tolist() == [[0, 1, 2]] and r.lengths.tolist() == m.tolist() and r.tokens.tolist() == [[1, 1, 1]]


def test_captured_and_replayed():
    logits, scores = _random(5, 4, 3001, torch.float32)
    state = torch.randn(2, 5, 4, 33, device="cuda")
    call = lambda: ak.ak_beam_reorder(state, ak.ak_beam_select(logits, scores).parents, dim=1)  # noqa: E731
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for seed in range(3):
        logits.copy_(_random(5, 4, 3001, torch.float32, 40 + seed)[0])
        was = state.clone()
        g.replay()
        p = ak.ak_beam_select(logits, scores).parents.long()
        assert torch.equal(state, was.gather(2, p[None, :, :, None].expand_as(was)))


@pytest.mark.parametrize("k", [1, 2, 4, 5, 8, 16, 23, 32])
@pytest.mark.parametrize("dtype,width", [(torch.float32, 64), (torch.float32, 7), (torch.bfloat16, 33), (torch.uint8, 13),
                                         (torch.int64, 1500), (torch.float32, 1)])
def test_reorder(k, dtype, width):
    g = torch.Generator().manual_seed(k)
    state = torch.randint(0, 100, (3, 5, k, width), generator=g).to(dtype).cuda()
    parents = torch.randint(-1, k + 1, (5, k), generator=g, dtype=torch.int32)
    parents[0] = torch.arange(k)
    parents[1] = torch.arange(k).flip(0)
    parents[2] = k - 1
    want = state.clone()
    for r in range(5):
        for j in range(k):
            if 0 <= int(parents[r, j]) < k:
                want[:, r, j] = state[:, r, int(parents[r, j])]
    assert torch.equal(ak.ak_beam_reorder(state, parents.cuda(), dim=1), want)


def test_reorder_of_views():
    big = torch.arange(4 * 6 * 3 * 50, device="cuda", dtype=torch.float32).reshape(4, 6, 3, 50)
    part = big[:, :, :, 10:40]
    parents = torch.tensor([[2, 2, 0]] * 6, dtype=torch.int32, device="cuda")
    want = big.clone()
    want[:, :, :, 10:40] = big[:, :, [2, 2, 0], 10:40]
    ak.ak_beam_reorder(part, parents, dim=1)
    assert torch.equal(big, want)
    one = torch.arange(6, device="cuda").reshape(2, 3)
    ak.ak_beam_reorder(one, parents[:2])
    assert one.tolist() == [[2, 2, 0], [5, 5, 3]]
    beams_first = torch.arange(24, device="cuda").reshape(3, 2, 4)  # [beams, requests, ...]
    ak.ak_beam_reorder(beams_first.transpose(0, 1), parents[:2])
    assert beams_first[:, 0, 0].tolist() == [16, 16, 0]
