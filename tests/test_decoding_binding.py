"""What the decoding operators' binding makes of gradients, of what it changes in place and of numbers out of range, on
the host."""
from __future__ import annotations

import pytest
import torch

import mapreduce_prefix_scan_gb300 as ak
from test_decoding_abi import L, _calls  # noqa: F401
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


WRITTEN = {
    "ak_gated_recurrence": {"out", "state_out"}, "ak_gated_recurrence_backward": {"dx", "dgate", "dstate"},
    "ak_gated_recurrence_step": {"state", "out"}, "ak_beam_select": {"out"}, "ak_beam_reorder": {"state"}, "ak_blocks_count": {"out"},
    "ak_blocks_fork": {"out"}, "ak_blocks_free": {"out", "counts"}, "ak_blocks_compact": {"out", "pairs", "counts"},
    "ak_blocks_copy": {"cache"},
}


@pytest.mark.parametrize("call", WRITTEN)
def test_autograd_learns_of_what_a_call_changes(host, call):  # noqa: F811
    """A tensor's version counts its changes, and counts no reading."""
    library = host(_Library())
    tensors, rest = _calls()[call]
    tensors = {n: _cuda(t) for n, t in tensors.items() if n != "workspace"}
    i32 = lambda *s: _cuda(torch.zeros(s, dtype=torch.int32))  # noqa: E731
    if call == "ak_beam_select":
        tensors["out"] = ak.BeamStep(_cuda(torch.zeros(2, 3)), i32(2, 3), i32(2, 3), _cuda(torch.zeros(2, 3, dtype=torch.bool)), i32(2, 3))
    if call == "ak_blocks_fork":
        tensors["out"] = ak.BlockFork(i32(5, 4), i32(5), i32(9), i32(5, 2), i32(1))
    before = {n: [u._version for u in (t if isinstance(t, tuple) else (t,))] for n, t in tensors.items()}
    getattr(ak, call)(**tensors, **rest)
    assert library.calls.pop(call)
    for n, t in tensors.items():
        for u, was in zip(t if isinstance(t, tuple) else (t,), before[n]):
            assert (u._version > was) == (n in WRITTEN[call]), n


@pytest.mark.parametrize("change", [
    lambda s: ak.ak_gated_recurrence_step(_cuda(torch.zeros(4, 3)), _cuda(torch.zeros(4, 3)), s),
    lambda s: ak.ak_gated_recurrence(_cuda(torch.zeros(4, 3)), _cuda(torch.zeros(4, 3)), out=s),
    lambda s: ak.ak_beam_reorder(s.view(2, 2, 3), _cuda(torch.zeros(2, 2, dtype=torch.int32))),
    lambda s: ak.ak_blocks_copy(s, _cuda(torch.zeros(2, 2, dtype=torch.int32))),
])
def test_a_backward_pass_over_what_has_changed_since_raises(host, change):  # noqa: F811
    host(_Library())
    state, w = _cuda(torch.ones(4, 3)), torch.ones(4, 3, requires_grad=True)
    loss = (w * state).sum()
    change(state)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()


def test_workspaces_can_be_sized(host, L):  # noqa: F811
    """What the queries answer is what the calls take, to the byte."""
    fork, compact = ak.ak_blocks_fork_workspace_size(5, 9), ak.ak_blocks_compact_workspace_size(9)
    assert fork >= 4 * (2 * 9 + 5) and compact >= 4 * (2 * 4 + 9)
    with pytest.raises(ak.AkError):
        ak.ak_blocks_fork_workspace_size(-1, 9)
    with pytest.raises(ak.AkError):
        ak.ak_blocks_compact_workspace_size(-1)
    for call, size in (("ak_blocks_fork", fork), ("ak_blocks_compact", compact)):
        library = host(_Library(sizes=size))
        tensors, rest = _calls()[call]
        tensors = {n: _cuda(t) for n, t in tensors.items()}
        getattr(ak, call)(**dict(tensors, workspace=_cuda(torch.zeros(size, dtype=torch.uint8))), **rest)
        assert library.calls.pop(call)
        with pytest.raises(ValueError, match="workspace"):
            getattr(ak, call)(**dict(tensors, workspace=_cuda(torch.zeros(size - 1, dtype=torch.uint8))), **rest)
        assert not library.calls
