"""Refusals of the gated recurrence, beam search and block operators: decided on the host, before anything touches a device."""
from __future__ import annotations

import ctypes

import pytest
import torch

import mapreduce_prefix_scan_gb300 as ak
from test_sequence_binding import STREAM_OF, _Cuda, _Library, _OtherCuda, _cuda, host  # noqa: F401
from mapreduce_prefix_scan_gb300 import sequence


@pytest.fixture(scope="module")
def L():
    from mapreduce_prefix_scan_gb300 import build
    build.build()
    from mapreduce_prefix_scan_gb300 import _abi
    return _abi.load()


R = ctypes.byref


def _shape(**kw):
    from mapreduce_prefix_scan_gb300._abi import ak_recurrence
    a = ak_recurrence(100, 2, 64, 2, 0)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def test_recurrence_refusals(L):
    from mapreduce_prefix_scan_gb300._abi import AK_ERR_INVALID_ARG as INV, AK_ERR_UNSUPPORTED as UNS, ak_recurrence, ak_rows
    assert ctypes.sizeof(ak_rows) == 16 and ctypes.sizeof(ak_recurrence) == 32
    H = lambda p=0x10000, t=64: ak_rows(p, t)  # noqa: E731

    def fwd(a=None, x=H(), g=H(), h=H(), off=0x2000, s0=None, s1=None):
        return L.ak_gated_recurrence(R(a or _shape()), R(x), R(g), off, s0, R(h), s1, None, None)

    shapes = (dict(tokens=-1), dict(seqs=-1), dict(channels=0), dict(channels=1 << 40), dict(dtype=99), dict(dtype=-1), dict(form=2),
              dict(form=-1), dict(tokens=1 << 40), dict(seqs=1 << 40))
    for bad in shapes:
        assert fwd(_shape(**bad)) == INV, bad
    assert fwd(_shape(dtype=1)) == UNS and fwd(_shape(dtype=3)) == UNS
    for bad in (dict(x=H(0)), dict(g=H(0x10001)), dict(x=H(t=-1)), dict(h=H(t=0)), dict(h=H(t=63)), dict(h=H(0)), dict(off=None),
                dict(off=0x2002), dict(s0=0x3001), dict(s1=0x3002)):
        assert fwd(**bad) == INV, bad
    assert L.ak_gated_recurrence(None, R(H()), R(H()), 0x2000, None, R(H()), None, None, None) == INV
    assert L.ak_gated_recurrence(R(_shape()), None, R(H()), 0x2000, None, R(H()), None, None, None) == INV
    assert fwd(_shape(tokens=0)) == 0  # nothing to do

    def bwd(a=None, dh=H(), x=H(), g=H(), h=H(), dx=H(), dg=H(), s0=None, ds=None, d0=None):
        return L.ak_gated_recurrence_backward(R(a or _shape(form=1)), R(dh), R(x), R(g), R(h), 0x2000, s0, ds, R(dx), R(dg), d0, None, None)

    for bad in shapes:
        assert bwd(_shape(**bad)) == INV, bad
    for bad in (dict(dh=H(0)), dict(x=H(0)), dict(g=H(t=-1)), dict(h=H(0x10001)), dict(dx=H(t=0)), dict(dg=H(t=10)), dict(s0=0x3001),
                dict(ds=0x3002), dict(d0=0x3003)):
        assert bwd(**bad) == INV, bad

    def step(a=None, x=H(), g=H(), state=0x4000, slots=0x5000, ns=5, h=H()):
        return L.ak_gated_recurrence_step(R(a or _shape()), R(x), R(g), state, slots, ns, R(h), None, None)

    for bad in (dict(state=None), dict(state=0x4002), dict(slots=0x5001), dict(ns=-1), dict(h=H(t=0)), dict(x=H(0)),
                dict(a=_shape(form=7)), dict(a=_shape(tokens=1 << 30, channels=1 << 30))):
        assert step(**bad) == INV, bad
    assert step(_shape(tokens=0)) == 0


def test_beam_refusals(L):
    from mapreduce_prefix_scan_gb300._abi import AK_ERR_INVALID_ARG as INV, AK_ERR_UNSUPPORTED as UNS
    good = dict(x=0x1000, bs=400, ks=100, dt=0, n=2, k=4, v=100, keep=4, s=0x2000, d=0x3001, m=0x4000, end=5, pen=0.5, os=0x5000,
                ot=0x6000, op=0x7000, od=0x8001, ol=0x9000)

    def call(**kw):
        return L.ak_beam_select(*dict(good, **kw).values(), None, None)

    for bad in (dict(x=None), dict(x=0x1002), dict(bs=-1), dict(ks=-1), dict(dt=44), dict(n=-1), dict(n=1 << 40), dict(k=0), dict(k=33),
                dict(v=0), dict(v=1 << 40), dict(keep=0), dict(keep=33), dict(s=None), dict(s=0x2001), dict(m=0x4001), dict(end=-2),
                dict(end=100), dict(pen=float("nan")), dict(pen=float("inf")), dict(os=None), dict(ot=None), dict(op=None),
                dict(ot=0x6002), dict(ol=0x9001)):
        assert call(**bad) == INV, bad
    assert call(dt=1) == UNS and call(n=0) == 0

    good_r = dict(s=0x1000, o=2, os=4000, n=3, bs=1000, k=4, ks=200, b=200, p=0x2000)

    def reorder(**kw):
        return L.ak_beam_reorder(*dict(good_r, **kw).values(), None, None)

    for bad in (dict(s=None), dict(o=-1), dict(os=-1), dict(os=199), dict(n=-1), dict(bs=199), dict(k=0), dict(k=33), dict(ks=199),
                dict(ks=0), dict(b=-1), dict(p=None), dict(p=0x2002), dict(o=1 << 40), dict(n=1 << 40)):
        assert reorder(**bad) == INV, bad
    assert reorder(n=0) == 0 and reorder(b=0) == 0 and reorder(o=0) == 0


def test_block_refusals(L):
    from mapreduce_prefix_scan_gb300._abi import AK_ERR_INVALID_ARG as INV, AK_ERR_WORKSPACE as WS
    table = dict(t=0x1000, ts=8, w=8, m=0x2000, n=5)
    bad_table = (dict(t=None), dict(t=0x1002), dict(ts=7), dict(ts=0), dict(w=-1), dict(m=None), dict(n=-1), dict(n=1 << 40))

    def refuse(call, bad):
        for b in bad:
            assert call(**b) == INV, b

    def count(**kw):
        return L.ak_blocks_count(*dict(dict(table, b=16, nb=9, r=0x3000), **kw).values(), None, None)

    refuse(count, bad_table + (dict(b=0), dict(nb=-1), dict(nb=1 << 40), dict(r=None), dict(r=0x3001)))
    good_f = dict(table, p=0x2100, nn=6, f=0x2200, nf=3, b=16, nb=9, ot=0x4000, os=8, ol=0x5000, r=0x3000, pr=0x6000, c=0x7000, ws=0x8000, wb=1 << 20)

    def fork(**kw):
        return L.ak_blocks_fork(*dict(good_f, **kw).values(), None, None)

    refuse(fork, bad_table + (dict(p=None), dict(nn=-1), dict(nn=1 << 40), dict(f=None), dict(nf=-1), dict(b=-1), dict(nb=-1), dict(ot=None),
                              dict(ot=0x1000), dict(os=7), dict(ol=None), dict(ol=0x2000), dict(r=None), dict(pr=None), dict(c=None), dict(c=0x7001)))
    assert fork(ws=None) == WS and fork(wb=64) == WS and fork(ws=0x8004) == WS
    assert L.ak_blocks_free(None, 5, 0x1000, 0x2000, None, None) == INV
    assert L.ak_blocks_free(0x1000, -1, 0x1000, 0x2000, None, None) == INV
    assert L.ak_blocks_free(0x1000, 5, None, 0x2000, None, None) == INV
    assert L.ak_blocks_free(0x1000, 5, 0x1000, None, None, None) == INV
    good_c = dict(table, r=0x3000, b=16, nb=9, ot=0x4000, os=8, pr=0x6000, c=0x7000, ws=0x8000, wb=1 << 20)

    def compact(**kw):
        return L.ak_blocks_compact(*dict(good_c, **kw).values(), None, None)

    refuse(compact, bad_table + (dict(r=None), dict(b=0), dict(nb=-1), dict(ot=None), dict(os=7), dict(ot=0x1000, os=9), dict(pr=None), dict(c=None)))
    assert compact(ws=None) == WS and compact(wb=64) == WS
    good_y = dict(x=0x1000, o=2, os=9000, nb=9, bs=1000, i=1000, p=0x2000, np=4, c=0x3000)

    def copy(**kw):
        return L.ak_blocks_copy(*dict(good_y, **kw).values(), None, None)

    refuse(copy, (dict(x=None), dict(o=-1), dict(os=-1), dict(os=999), dict(nb=-1), dict(bs=999), dict(i=-1), dict(p=None), dict(p=0x2001),
                  dict(np=-1), dict(np=1 << 40), dict(c=0x3002)))
    assert copy(np=0) == 0 and copy(i=0) == 0 and copy(o=0) == 0 and copy(nb=0) == 0
    b = ctypes.c_size_t()
    assert L.ak_blocks_fork_workspace_size(10, 100, None, R(b)) == 0 and b.value >= 840
    assert L.ak_blocks_compact_workspace_size(100, None, R(b)) == 0 and b.value >= 800
    for f in (lambda: L.ak_blocks_fork_workspace_size(-1, 100, None, R(b)), lambda: L.ak_blocks_fork_workspace_size(1, 100, None, None),
              lambda: L.ak_blocks_compact_workspace_size(-1, None, R(b)), lambda: L.ak_blocks_compact_workspace_size(1, None, None)):
        assert f() == INV


# ---------------------------------------------------------------------------
# the binding, over host memory under a device's name
# ---------------------------------------------------------------------------


def _calls():
    """Each entry point with all of its tensor arguments by name."""
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    f32 = lambda *s: torch.zeros(s)  # noqa: E731
    ws = lambda: torch.zeros(8192, dtype=torch.uint8)  # noqa: E731
    xg = lambda: dict(x=f32(9, 8), gate=f32(9, 8))  # noqa: E731
    tl = lambda: dict(block_table=i32(3, 4), lens=i32(3))  # noqa: E731
    return {
        "ak_gated_recurrence": (dict(xg(), offsets=i32(3), state=f32(2, 8), out=f32(9, 8), state_out=f32(2, 8)), {}),
        "ak_gated_recurrence_backward": (dict(xg(), dh=f32(9, 8), h=f32(9, 8), offsets=i32(3), state=f32(2, 8), dstate_out=f32(2, 8),
                                              dx=f32(9, 8), dgate=f32(9, 8), dstate=f32(2, 8)), {}),
        "ak_gated_recurrence_step": (dict(xg(), state=f32(20, 8), slots=i32(9), out=f32(9, 8)), {}),
        "ak_beam_select": (dict(logits=f32(2, 3, 7), scores=f32(2, 3), done=torch.zeros(2, 3, dtype=torch.bool), lengths=i32(2, 3)), {}),
        "ak_beam_reorder": (dict(state=f32(4, 3, 5), parents=i32(4, 3)), {}),
        "ak_blocks_count": (dict(tl(), out=i32(9)), dict(block_size=4, blocks=9)),
        "ak_blocks_fork": (dict(tl(), parents=i32(5), free_blocks=i32(2), workspace=ws()), dict(block_size=4, blocks=9)),
        "ak_blocks_free": (dict(refs=i32(9), out=i32(9), counts=i32(1)), {}),
        "ak_blocks_compact": (dict(tl(), refs=i32(9), out=i32(3, 4), pairs=i32(4, 2), counts=i32(2), workspace=ws()), dict(block_size=4)),
        "ak_blocks_copy": (dict(cache=f32(9, 5), pairs=i32(4, 2), counts=i32(1)), {}),
    }


ARGUMENTS = [(call, name) for call, (tensors, _) in _calls().items() for name in tensors]


@pytest.mark.parametrize("call,name", ARGUMENTS)
def test_an_argument_on_another_device_is_refused(host, call, name):  # noqa: F811
    library = host(_Library())
    tensors, rest = _calls()[call]
    tensors = {n: _cuda(t) for n, t in tensors.items()}
    getattr(ak, call)(**tensors, **rest)
    assert library.calls.pop(call)
    for stray in (tensors[name].as_subclass(torch.Tensor), tensors[name].as_subclass(_OtherCuda)):
        with pytest.raises(ValueError):
            getattr(ak, call)(**dict(tensors, **{name: stray}), **rest)
    assert not library.calls


@pytest.mark.parametrize("call,name", ARGUMENTS)
def test_an_argument_of_another_type_is_refused(host, call, name):  # noqa: F811
    library = host(_Library())
    tensors, rest = _calls()[call]
    tensors = {n: _cuda(t) for n, t in tensors.items()}
    if name in ("workspace", "cache") or (call, name) == ("ak_beam_reorder", "state"):
        return  # of any type
    with pytest.raises(ValueError):
        getattr(ak, call)(**dict(tensors, **{name: _cuda(tensors[name].as_subclass(torch.Tensor).to(torch.int16))}), **rest)
    assert not library.calls


@pytest.mark.parametrize("call", _calls())
@pytest.mark.parametrize("current,refused", [(0, False), (1, True)])
def test_tensors_of_a_device_that_is_not_current_are_refused(host, monkeypatch, call, current, refused):  # noqa: F811
    library = host(_Library())
    monkeypatch.setattr(sequence, "_stream_of", STREAM_OF)
    monkeypatch.setattr(sequence, "_device", lambda: current)
    tensors, rest = _calls()[call]
    tensors = {n: _cuda(t) for n, t in tensors.items()}
    if refused:
        with pytest.raises(ValueError, match="current CUDA device"):
            getattr(ak, call)(**tensors, **rest, stream=7)
    else:
        getattr(ak, call)(**tensors, **rest, stream=7)
    assert (call in library.calls) != refused


def test_shapes_that_would_be_read_in_the_wrong_order_are_refused(host):  # noqa: F811
    library = host(_Library())
    for call, name, shape in (("ak_gated_recurrence", "gate", (8, 9)), ("ak_gated_recurrence", "state", (8, 2)),
                              ("ak_gated_recurrence_backward", "h", (8, 9)), ("ak_gated_recurrence_step", "state", (16, 10)),
                              ("ak_beam_select", "scores", (3, 2)), ("ak_beam_select", "done", (6,)), ("ak_beam_reorder", "parents", (3, 4)),
                              ("ak_blocks_copy", "pairs", (2, 4)), ("ak_blocks_compact", "pairs", (2, 4))):
        tensors, rest = _calls()[call]
        tensors = {n: _cuda(t) for n, t in tensors.items()}
        with pytest.raises(ValueError):
            getattr(ak, call)(**dict(tensors, **{name: tensors[name].reshape(shape)}), **rest)
    x = _cuda(torch.zeros(9, 16))
    with pytest.raises(ValueError):
        ak.ak_gated_recurrence(x[:, ::2], x[:, ::2])
    with pytest.raises(ValueError):
        ak.ak_gated_recurrence(x, x, form="other")
    with pytest.raises(ValueError):
        ak.ak_gated_recurrence(x, x, offsets=_cuda(torch.zeros(0, dtype=torch.int32)))
    with pytest.raises(ValueError):
        ak.ak_gated_recurrence_step(x, x, _cuda(torch.zeros(8, 16)))
    with pytest.raises(ValueError):
        ak.ak_beam_reorder(_cuda(torch.zeros(4, 3, 5, 2)).transpose(2, 3), _cuda(torch.zeros(4, 3, dtype=torch.int32)))
    assert not library.calls


def test_in_place_operators_do_not_pass_for_differentiable(host):  # noqa: F811
    library = host(_Library())
    t = _cuda(torch.zeros(4, 3, 5)).requires_grad_()
    with pytest.raises(RuntimeError, match="gradient"):
        ak.ak_beam_reorder(t, _cuda(torch.zeros(4, 3, dtype=torch.int32)))
    with pytest.raises(RuntimeError, match="gradient"):
        ak.ak_blocks_copy(t, _cuda(torch.zeros(2, 2, dtype=torch.int32)))
    assert not library.calls


def test_views_are_handed_over_as_they_lie(host):  # noqa: F811
    library = host(_Library())
    cache = _cuda(torch.zeros(3, 2, 30, 8, 16))  # [layer, k or v, block, ...]
    pairs = _cuda(torch.zeros(4, 2, dtype=torch.int32))
    ak.ak_blocks_copy(cache, pairs, dim=2)
    assert library.calls["ak_blocks_copy"][1:6] == (6, 30 * 512, 30, 512, 512)
    ak.ak_blocks_copy(cache[:, 0], pairs, dim=1)
    assert library.calls["ak_blocks_copy"][1:6] == (3, 60 * 512, 30, 512, 512)
    state = _cuda(torch.zeros(4, 6, 3, 10))
    ak.ak_beam_reorder(state[..., 2:7], _cuda(torch.zeros(6, 3, dtype=torch.int32)), dim=1)
    assert library.calls["ak_beam_reorder"][1:8] == (4, 720, 6, 120, 3, 40, 20)
