"""Where a NaN or an infinity goes, against the recurrence in 64 bits: the same results are not finite, and the others
keep their bounds (those of test_linear_attention_gpu)."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import mapreduce_prefix_scan_gb300 as ak
from sequence_reference import attention, attention_gradients
from test_linear_attention_gpu import DT, _bound, _dev, _inputs, _off

pytestmark = pytest.mark.gpu

LENS = [70, 129, 0, 64]
LD = [-0.3, 0.0, -3.0]  # at the last one, weights over a chunk underflow


def _same(got, want, bound, name):
    got = got.double().cpu().numpy()
    assert np.array_equal(np.isfinite(got), np.isfinite(want)), name
    ok = np.isfinite(want)
    err, tol = np.abs(got - want)[ok], bound[ok] + 1e-30
    assert (err <= tol).all(), f"{name}: worst ratio {np.max(err / tol):.3g}"


# a sequence's first token, the last and first of chunks, the last of a sequence; a whole chunk and a short one
PLACES = [("v", 0), ("v", 40), ("v", 63), ("v", 64), ("v", 69), ("v", 70 + 63), ("v", 70 + 64), ("v", 70 + 128), ("v", 199),
          ("k", 40), ("k", 66), ("k", 70 + 64), ("k", 70 + 128), ("q", 40), ("q", 70 + 128), ("do", 40), ("do", 70 + 64),
          ("s0", 1), ("ds", 1)]


@pytest.mark.parametrize("dtype,dim", [("bf16", 64), ("bf16", 128), ("bf16", 80), ("f32", 64)])
@pytest.mark.parametrize("windows", [1, 3])
@pytest.mark.parametrize("what,at", PLACES)
@pytest.mark.parametrize("value", [np.nan, -np.inf])
def test_only_what_the_recurrence_reaches(dtype, dim, windows, what, at, value):
    q, k, v, do, ld, off, s0, ds = _inputs(at, dtype, LENS, 3, dim, dim, ld=LD)
    x = dict(q=q, k=k, v=v, do=do, s0=s0, ds=ds)
    for h in range(3):
        x[what][(at, h, 5 + h) + ((7 + h,) if what in ("s0", "ds") else ())] = value
    a = {n: np.abs(y) for n, y in x.items()}
    d, opts = DT[dtype], dict(target_blocks=windows)
    with np.errstate(all="ignore"):
        want, sf, mass = attention(q, k, v, ld, off, s0, 0.37)
        _, sa, _ = attention(a["q"], a["k"], a["v"], ld, off, a["s0"])
        grads = attention_gradients(do, q, k, v, ld, off, s0, ds, 0.37)
        gmass = attention_gradients(a["do"], a["q"], a["k"], a["v"], ld, off, a["s0"], a["ds"], 0.37)
        o, s1 = ak.ak_linear_attention(_dev(q, d), _dev(k, d), _dev(v, d), _dev(ld), offsets=_off(off), state=_dev(s0),
                                       scale=0.37, final_state=True, opts=opts)
        _same(o, want, _bound(dtype, LENS, dim, want, mass), "o")
        _same(s1, sf, _bound("f32", LENS, dim, sf, sa), "state")
        got = ak.ak_linear_attention_backward(_dev(do, d), _dev(q, d), _dev(k, d), _dev(v, d), _dev(ld), offsets=_off(off),
                                              state=_dev(s0), dstate_out=_dev(ds), scale=0.37, opts=opts)
        for i, name in enumerate(("dq", "dk", "dv", "dstate")):
            _same(got[i], grads[i], _bound(dtype if i < 3 else "f32", LENS, dim, grads[i], gmass[i]), name)


@pytest.mark.parametrize("dim", [64, 128])
def test_scores_beyond_the_type_stay_with_later_tokens(dim):
    """Finite q and k whose product is not: k of token 20 times q of token 10, which comes before it, is masked."""
    q, k, v, _, ld, off, _, _ = _inputs(3, "bf16", [64], 1, dim, dim, state=False, ld=[-0.1])
    q[10, 0], k[20, 0] = 2.0**66, 2.0**66
    q[21:, 0, :] = 0
    o, _ = ak.ak_linear_attention(_dev(q, torch.bfloat16), _dev(k, torch.bfloat16), _dev(v, torch.bfloat16), _dev(ld))
    want, _, mass = attention(q, k, v, ld, off, None)
    keep = [t for t in range(64) if t < 20]
    got = o.double().cpu().numpy()[keep]
    assert np.isfinite(got).all()
    assert (np.abs(got - want[keep]) <= _bound("bf16", [64], dim, want, mass)[keep]).all()
