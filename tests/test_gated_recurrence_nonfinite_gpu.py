"""Single tokens on states that are not finite."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import decoding_reference as ref
import mapreduce_prefix_scan_gb300 as ak

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("channels", [13, 64])  # rows of odd and of whole vectors
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("form", ["decay", "gate"])
def test_a_step_keeps_an_infinite_state(form, dtype, channels):
    """a h + b x in 64 bits says what an infinite h gives: itself at every a above 0, NaN beside the other infinity and at a = 0."""
    inf, nan = float("inf"), float("nan")
    gates = [-20.0, -2.0, -0.6, -1e-3, 0.0, 3.0, 30.0] + ([inf] if form == "gate" else [-inf])
    rows = [(g, h, x) for g in gates for h in (inf, -inf, nan, 2.0) for x in (1.5, -0.0, inf, -inf, nan)]
    fill = lambda i, t: torch.tensor([r[i] for r in rows], dtype=t)[:, None].repeat(1, channels).cuda()  # noqa: E731
    gate, state, x = fill(0, dtype), fill(1, torch.float32), fill(2, dtype)
    a, b = ref.weights(gate.double().cpu().numpy(), form)
    with np.errstate(invalid="ignore"):
        want = a * state.double().cpu().numpy() + b * x.double().cpu().numpy()
    h = ak.ak_gated_recurrence_step(x, gate, state, form=form)
    for got in (h, state):
        got = got.double().cpu().numpy()
        wild = ~np.isfinite(want)
        assert np.array_equal(got[wild], want[wild], equal_nan=True)
        assert np.isfinite(got[~wild]).all()
