"""Paths of linear attention that long or many sequences take, against the recurrence in 64 bits with the bounds of
test_linear_attention_gpu, and the precision of the states that include/ak.h states."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import mapreduce_prefix_scan_gb300 as ak
from sequence_reference import attention, attention_gradients
from test_linear_attention_gpu import DT, _bound, _close, _dev, _inputs, _mass_gradients, _off

pytestmark = pytest.mark.gpu


def _check(dtype, lens, h, dim, ld, heads=None, state=True, seed=0, lo=0, extra=0, **kw):
    """Forward and backward calls of `h` heads; `heads` of them (all) against the recurrence. `lo` tokens before and
    `extra` after the sequences hold NaN."""
    q, k, v, do, ld, off, s0, ds = _inputs(seed, dtype, lens, h, dim, dim, state, ld)
    d, scale, pick = DT[dtype], 0.37, list(range(h)) if heads is None else heads
    t = sum(lens)
    grow = lambda x: torch.cat([torch.full((n,) + x.shape[1:], float("nan"), device="cuda", dtype=d) if n else y
                                for n, y in ((lo, None), (None, _dev(x, d)), (extra, None)) if n != 0])
    call = dict(offsets=_off(off + lo), state=_dev(s0), scale=scale, **kw)
    o, s1 = ak.ak_linear_attention(grow(q), grow(k), grow(v), _dev(ld), final_state=True, **call)
    g = ak.ak_linear_attention_backward(grow(do), grow(q), grow(k), grow(v), _dev(ld), dstate_out=_dev(ds), **call)
    some = lambda x: None if x is None else x[:, pick]
    q, k, v, do, s0, ds, ld = some(q), some(k), some(v), some(do), some(s0), some(ds), ld[pick]
    want, sf, mass = attention(q, k, v, ld, off, s0, scale)
    _, sa, _ = attention(*(np.abs(x) for x in (q, k, v)), ld, off, None if s0 is None else np.abs(s0))
    for x in (o, *g[:3]):
        assert (x[:lo] == 0).all() and (x[lo + t:] == 0).all()
    _close(o[lo:lo + t, pick], want, _bound(dtype, lens, dim, want, mass), "o")
    _close(s1[:, pick], sf, _bound("f32", lens, dim, sf, sa), "state")
    want = attention_gradients(do, q, k, v, ld, off, s0, ds, scale)
    mass = _mass_gradients(do, q, k, v, ld, off, s0, ds, scale)
    for i, name in enumerate(("dq", "dk", "dv")):
        _close(g[i][lo:lo + t, pick], want[i], _bound(dtype, lens, dim, want[i], mass[i]), name)
    if state:
        _close(g[3][:, pick], want[3], _bound("f32", lens, dim, want[3], mass[3]), "dstate")


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("lens", [[1100], [2200], [37, 1500, 1]])
def test_frames_of_the_state(dim, lens):
    """One window: the state is kept divided by the decay for 16, 16, 7, 2 and 1 chunks, or scaled in every chunk, and
    the walk passes the ends of several such frames. The first head grows."""
    _check("bf16", lens, 7, dim, [0.004, -0.0, -0.0293, -0.0656, -0.1875, -0.3125, -0.6], opts=dict(target_blocks=1))


@pytest.fixture
def by_sequence(capfd, monkeypatch):
    """Switches the log on; the value says whether every call since took a block for each sequence."""
    monkeypatch.setenv("AK_LOG", "1")

    def all_of_them():
        lines = [x for x in capfd.readouterr().err.splitlines() if "linear_attention" in x]
        assert lines
        return all("a block each" in x for x in lines)
    return all_of_them


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens", [[30, 100, 0, 100, 70], [0, 70, 0, 70, 120, 0], [1, 2, 257]])
@pytest.mark.parametrize("lo,extra", [(0, 0), (3, 15)])
def test_blocks_ranked_by_length(by_sequence, dtype, lens, lo, extra):
    """A block for each sequence, the longest first: unsorted lengths with ties and empty ones, and tokens of no sequence
    before and after them."""
    _check(dtype, lens, 2, 64, None, lo=lo, extra=extra)
    assert by_sequence()


@pytest.mark.parametrize("dim", [64, 128])
def test_long_sequences_ranked(by_sequence, dim):
    _check("bf16", [300, 40, 300, 0, 520, 64, 300, 129], 64, dim, None, heads=[0, 17, 63], max_len=520)
    assert by_sequence()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_more_sequences_than_blocks_sort(by_sequence, dtype):
    rng = np.random.default_rng(4)
    _check(dtype, rng.integers(0, 71, 300).tolist(), 2, 64, None, max_len=70)
    assert by_sequence()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens", [[300, 20, 0, 90], [40] * 40 + [400]])
def test_a_bound_on_the_lengths_that_is_too_small(dtype, lens):
    """max_len only guides how the token axis is cut."""
    _check(dtype, lens, 2, 64, None, max_len=10)


def test_more_sequences_than_a_grid_takes():
    """70000 sequences, most of them empty: windows of the token axis, states passed on."""
    rng = np.random.default_rng(5)
    n, h, d = 70000, 2, 8
    lens = (rng.random(n) < 0.01).astype(np.int64)
    off = np.concatenate([[0], np.cumsum(lens)])
    t = int(off[-1])
    q, k, v = (torch.randn(t, h, d, device="cuda") for _ in range(3))
    ld = torch.tensor([-0.1, -2.0], device="cuda")
    s0 = torch.randn(n, h, d, d, device="cuda")
    o, s1 = ak.ak_linear_attention(q, k, v, ld, offsets=_off(off), state=s0, final_state=True)
    at = torch.tensor(np.flatnonzero(lens), device="cuda")
    new = s0[at].double() * torch.exp(ld.double())[:, None, None] + k.double()[..., :, None] * v.double()[..., None, :]
    want = s0.double()
    want[at] = new
    assert (s1[at].double() - new).abs().max() <= 8 * 2.0**-24 * new.abs().max()
    rest = torch.ones(n, dtype=torch.bool, device="cuda")
    rest[at] = False
    assert torch.equal(s1[rest], s0[rest])
    w = torch.einsum("thi,thij->thj", q.double(), new)
    m = torch.einsum("thi,thij->thj", q.double().abs(), new.abs())
    assert ((o.double() - w).abs() <= (d + 16) * 2.0**-24 * m).all()


# ---------------------------------------------------------------------------------------------------------------------
# precision of the states
# ---------------------------------------------------------------------------------------------------------------------

LD = [0.0, -1e-5, -1e-4, -1e-3, -1 / 256, -0.02, -0.1, -0.3, -1.0, -4.0]


def _state_error(x, want):
    return ((x[0].double() - want).pow(2).sum((1, 2)).sqrt() / want.pow(2).sum((1, 2)).sqrt()).tolist()


def _states(dtype, t, dim, opts, scale=0.37):
    """Relative errors, in norm and for each head, of the final state and of the initial state's gradient, on normal
    inputs."""
    torch.manual_seed(t + dim)
    h = len(LD)
    q, k, v, do = (torch.randn(t, h, dim, device="cuda").bfloat16() for _ in range(4))
    ld = torch.tensor(LD, device="cuda")
    age = torch.arange(t, device="cuda", dtype=torch.float64)
    terms = lambda x, y, w: torch.einsum("ht,thi,thj->hij", torch.exp(ld.double()[:, None] * w), x.double(), y.double())
    d = DT[dtype]
    q, k, v, do = (x.to(d) for x in (q, k, v, do))
    _, s = ak.ak_linear_attention(q, k, v, ld, final_state=True, opts=opts)
    g = ak.ak_linear_attention_backward(do, q, k, v, ld, scale=scale, dstate=torch.empty_like(s), opts=opts)[3]
    scale = float(np.float32(scale))
    return _state_error(s, terms(k, v, age.flip(0))), _state_error(g, scale * terms(q, do, age + 1))


def _stated(t, window):
    """include/ak.h: 4e-7, and 7.5e-9 for each token that the decay remembers within a window."""
    return [4e-7 + 7.5e-9 * min(t, window, 1 / -np.expm1(x) if x else np.inf) for x in LD]


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("t", [2, 17, 63, 64, 65, 130, 300, 1000])
def test_states_of_bf16_calls_are_as_precise_as_stated(dim, t):
    """Values in two parts instead of three leave 2.4e-6 of each term: up to 300 tokens, and at any length of a decay that
    forgets, the stated bound is below that."""
    for errors in _states("bf16", t, dim, dict(target_blocks=1)):
        for ld, e, most in zip(LD, errors, _stated(t, t)):
            assert e <= most, (ld, e, most)


@pytest.mark.parametrize("windows,longest", [(1, 16000), (16, 1024)])
def test_states_over_a_long_axis(windows, longest):
    """Without decay the loss grows with the window, and shorter windows bound it. A float32 call rounds each of t sums to
    nearest, by 2^-24 of the state at most and in no direction: 2^-24 sqrt(t) in norm."""
    for errors in _states("bf16", 16000, 64, dict(target_blocks=windows)):
        for ld, e, most in zip(LD, errors, _stated(16000, longest)):
            assert e <= most, (ld, e, most)
    for errors in _states("f32", 16000, 64, dict(target_blocks=windows)):
        assert max(errors) <= 2.0**-24 * 16000**0.5
