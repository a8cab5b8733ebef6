"""The speculative-decoding example: all sequence operators in one loop."""
from __future__ import annotations

import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu


def _example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "speculative_decode.py")
    spec = importlib.util.spec_from_file_location("speculative_decode", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_states_and_log_agree_with_a_recomputation(dtype):
    r = _example().run(requests=9, rounds=6, drafts=3, dtype=dtype)
    assert 0 < r["kept"] < r["proposed"]
    assert all(6 <= m <= 24 for m in r["lengths"]) and sum(r["lengths"]) == r["kept"] + 9 * 6
    # every logged token was written, the first one of each request is where it began
    for h, f in zip(r["history"], r["first"].tolist()):
        assert (h >= 0).all() and int(h[0]) == f
    # no block belongs to two requests, none of the free ones is in a table
    used = r["table"][r["table"] >= 0].tolist()
    assert len(set(used)) == len(used) and not set(used) & set(r["free"].tolist())
    # states: float32 sums of up to 24 tokens' terms in two orders, each term rounded at most 24 + 16 times
    a, b = r["state"].double(), r["again"].double()
    assert float((a - b).abs().max()) <= 80 * 2.0**-24 * float(b.abs().max()) * 24
