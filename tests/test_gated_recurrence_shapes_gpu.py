"""The recurrence at the shapes that take its other kernels: long runs of rows at odd addresses, and clusters that are
smaller than the tiles of the token axis, down to one block that walks it alone."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import decoding_reference as ref
import mapreduce_prefix_scan_gb300 as ak
from test_gated_recurrence_gpu import HALF, _case, _close, _np, units

pytestmark = pytest.mark.gpu

SHAPES = {
    # 32 groups of channels x 20 tiles and more: the kernels of long runs
    "long runs": (1001, [1700, 1, 0, 3, 1293, 2003], 0, 0),
    "long runs, rows outside": (1001, [1700, 1, 0, 3, 1293, 1003], 301, 777),
    # clusters of two blocks, of one block (more groups of channels than clusters of two fit)
    "two blocks": (4096, [900, 0, 601, 2, 800], 0, 0),
    "one block": (8192, [299, 0, 1, 400], 0, 0),
    "one block, rows outside": (8191, [299, 0, 1, 400], 3, 130),
}


# A factor below 2^-126 is taken as 0 (the exponential's instruction gives no smaller ones), which is off by less than
# 2^-126 of what it is multiplied with: once a token, a run, a tile and a cluster's step. In five million values some gate
# of a few is as low as that, and a gradient of 2e-37 comes out as 0.
FLUSH = 4 * 2.0**-126


def _check(c, form, h, sf, grads):
    """The bounds of test_gated_recurrence_gpu.py, with what flushed factors add."""
    dtype, x, gate, off = c["x"].dtype, _np(c["x"]), _np(c["gate"]), c["off"]
    e, half = units(len(x), dtype), HALF[dtype]
    want, wsf, mass = ref.recurrence(x, gate, off, _np(c["s0"]), form)
    most = max(mass.max(), np.abs(_np(c["s0"])).max())
    _close(h, want, e * mass + half * (np.abs(want) + e * mass) + FLUSH * most, "h")
    ends = np.array([mass[off[i + 1] - 1] if off[i + 1] > off[i] else np.zeros(want.shape[1]) for i in range(len(wsf))])
    _close(sf, wsf, e * ends + FLUSH * most, "state")
    dx, dg, d0, gm, hm = ref.recurrence_gradients(_np(c["dh"]), x, gate, off, _np(c["s0"]), _np(c["ds"]), form)
    a, b = ref.weights(gate, form)
    top = max(gm.max(), np.abs(_np(c["ds"])).max())
    _close(grads[0], dx, b * (e * gm) + half * (np.abs(dx) + e * gm) + FLUSH * top, "dx")
    he = (2 * e + half) * hm
    ab = a if form == "decay" else a * b
    d = hm if form == "decay" else hm + np.abs(x)
    _close(grads[1], dg, ab * (gm * he + 2 * e * gm * d) + half * np.abs(dg) * (1 + 1e-2) + 2 * FLUSH * top * d.max(), "dgate")
    first = np.array([gm[off[i]] * a[off[i]] if off[i + 1] > off[i] else np.abs(d0[i]) for i in range(len(d0))])
    _close(grads[2], d0, e * first + FLUSH * top, "dstate")


def _apart(t, start):
    """The same values in rows that begin at odd addresses: a width and an offset of their own."""
    wide = torch.zeros(t.shape[0], t.shape[1] + 6 + (t.shape[1] + 1) % 2, dtype=t.dtype, device=t.device)
    view = wide[:, start: start + t.shape[1]]
    view.copy_(t)
    assert view.stride(0) % 2 == 1
    return view


@pytest.mark.parametrize("odd", [False, True])
@pytest.mark.parametrize("form", ["decay", "gate"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("name", SHAPES)
def test_forward_and_gradients(name, dtype, form, odd):
    channels, lens, before, after = SHAPES[name]
    c = _case(lens, channels, dtype, form, seed=channels + len(lens), before=before, after=after)
    for t in ("x", "gate", "dh"):
        c[t][:before] = float("nan")  # rows outside every sequence hold anything
        c[t][before + sum(lens):] = float("inf")
    ins = {t: _apart(c[t], 1 + i) if odd else c[t] for i, t in enumerate(("x", "gate", "dh"))}
    h, sf = ak.ak_gated_recurrence(ins["x"], ins["gate"], form=form, offsets=c["offsets"], state=c["s0"], final_state=True)
    grads = ak.ak_gated_recurrence_backward(ins["dh"], ins["x"], ins["gate"], _apart(h, 3) if odd else h, form=form, offsets=c["offsets"],
                                            state=c["s0"], dstate_out=c["ds"])
    for t in (h, *grads[:2]):
        assert not t[:before].any() and not t[before + sum(lens):].any()
    # where a row lies does not show (in runs that hold rows outside every sequence, what those hold may, in the rounding)
    if odd:
        same = dict(form=form, offsets=c["offsets"], state=c["s0"])
        plain = ak.ak_gated_recurrence(c["x"], c["gate"], final_state=True, **same)
        assert torch.equal(h, plain[0]) and torch.equal(sf, plain[1])
        # in place, states too
        x, s = ins["x"], c["s0"].clone()
        ak.ak_gated_recurrence(x, ins["gate"], form=form, offsets=c["offsets"], state=s, out=x, state_out=s)
        assert torch.equal(x, h) and torch.equal(s, sf)
        assert not x._base[:, :1].any()
    for t in ("x", "gate", "dh"):
        c[t][:before] = 0
        c[t][before + sum(lens):] = 0
    _check(c, form, h, sf, grads)
