"""What the decoding operators' binding makes of gradients, of what it changes in place and of numbers out of range, on
the host."""
from __future__ import annotations

import pytest
import torch

import mapreduce_prefix_scan_gb300 as ak
from test_decoding_abi import _calls
from test_sequence_binding import _Library, _cuda, host  # noqa: F401


@pytest.mark.parametrize("asks", ["logits", "scores"])
@pytest.mark.parametrize("given", [False, True])
def test_a_beam_step_does_not_pass_for_differentiable(host, asks, given):  # noqa: F811
    """Its scores are no constants: a backward pass through them is an error, not a gradient of nothing."""
    library = host(_Library())
    tensors, _ = _calls()["ak_beam_select"]
    tensors = {n: _cuda(t) for n, t in tensors.items()}
    tensors[asks].requires_grad_()
    out = ak.BeamStep(*(_cuda(torch.zeros(2, 3, dtype=d)) for d in (torch.float32, torch.int32, torch.int32, torch.bool, torch.int32)))
    step = ak.ak_beam_select(**tensors, out=out if given else None)
    assert isinstance(step, ak.BeamStep) and library.calls.pop("ak_beam_select")
    assert not any(t.requires_grad for t in step[1:])
    with pytest.raises(RuntimeError, match="no gradient"):
        step.scores.sum().backward()
    if given:
        assert all(a.data_ptr() == b.data_ptr() for a, b in zip(step, out))
    with torch.no_grad():
        assert not ak.ak_beam_select(**tensors).scores.requires_grad
    assert not ak.ak_beam_select(**{n: t.detach() for n, t in tensors.items()}).scores.requires_grad


@pytest.mark.parametrize("call,name,value", [("ak_beam_select", "end_token", 3), ("ak_beam_select", "keep", 2), ("ak_blocks_count", "block_size", 4),
                                             ("ak_blocks_fork", "block_size", 4), ("ak_blocks_compact", "block_size", 4)])
def test_numbers_past_32_bits_are_refused(host, call, name, value):  # noqa: F811
    """ctypes hands over their low bits: 2^32 + 4 tokens a block would pass for 4."""
    library = host(_Library())
    tensors, rest = _calls()[call]
    tensors = {n: _cuda(t) for n, t in tensors.items()}
    getattr(ak, call)(**tensors, **dict(rest, **{name: value}))
    assert library.calls.pop(call)
    for far in (1 << 32, -(1 << 32), 1 << 63):
        with pytest.raises(ValueError, match=name):
            getattr(ak, call)(**tensors, **dict(rest, **{name: value + far}))
    assert not library.calls
