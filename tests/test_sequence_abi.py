"""Refusals of the sequence operators' C entry points: decided on the host, before anything touches a device."""
from __future__ import annotations

import ctypes

import pytest


@pytest.fixture(scope="module")
def L():
    from mapreduce_prefix_scan_gb300 import build
    build.build()
    from mapreduce_prefix_scan_gb300 import _abi
    return _abi.load()


def test_structs(L):
    from mapreduce_prefix_scan_gb300 import _abi
    assert ctypes.sizeof(_abi.ak_heads) == 24 and ctypes.sizeof(_abi.ak_linattn) == 48


def test_batch_layout_refusals(L):
    from mapreduce_prefix_scan_gb300._abi import AK_ERR_INVALID_ARG as INV, AK_ERR_WORKSPACE as WS
    good = dict(ctx=0x1000, new=0x2000, n=10, table=0x3000, stride=8, width=8, free=0x4000, nfree=5, block=16, most=64,
                off=0x5000, slots=0x6000, pos=0x7000, req=0x8000, counts=0x9000, ws=None, wb=0)

    def call(**kw):
        a = dict(good, **kw)
        return L.ak_batch_layout(*a.values(), None, None)

    for bad in (dict(n=-1), dict(ctx=None), dict(new=None), dict(new=0x2002), dict(table=None), dict(stride=7),
                dict(width=-1), dict(nfree=-1), dict(free=None), dict(block=0), dict(block=-16), dict(most=-1),
                dict(off=None), dict(slots=None), dict(slots=0x6004), dict(pos=None), dict(req=0x8001), dict(counts=None),
                dict(n=1 << 40), dict(most=1 << 40)):
        assert call(**bad) == INV, bad
    assert call(n=5000) == WS
    b = ctypes.c_size_t()
    assert L.ak_batch_layout_workspace_size(5000, None, ctypes.byref(b)) == 0 and b.value > 5000 * 4
    assert L.ak_batch_layout_workspace_size(-1, None, ctypes.byref(b)) == INV
    assert L.ak_batch_layout_workspace_size(5, None, None) == INV
    assert call(n=5000, ws=0x10000, wb=b.value // 2) == WS
    assert call(n=5000, ws=0x10001, wb=1 << 20) == WS


def test_verify_drafts_refusals(L):
    from mapreduce_prefix_scan_gb300._abi import AK_ERR_INVALID_ARG as INV, AK_ERR_UNSUPPORTED as UNS
    good = dict(p=0x1000, pr=400, pw=100, q=0x2000, qr=300, qw=100, dt=0, d=0x3000, m=0x4000, u=0x5000, e=0x6000, es=100,
                n=2, k=3, v=100, t=0x7000, a=0x8000)

    def call(**kw):
        a = dict(good, **kw)
        return L.ak_verify_drafts(*a.values(), None, None)

    for bad in (dict(p=None), dict(p=0x1002), dict(pr=-1), dict(pw=-1), dict(q=0x2001), dict(qr=-1), dict(d=None), dict(u=None),
                dict(e=None), dict(es=-1), dict(n=-1), dict(k=-1), dict(v=0), dict(t=None), dict(a=0x8002), dict(m=0x4001),
                dict(dt=44), dict(n=1 << 40), dict(v=1 << 40)):
        assert call(**bad) == INV, bad
    assert call(dt=1) == UNS and call(dt=3) == UNS
    assert call(n=0) == 0  # nothing to do


def _linattn(**kw):
    from mapreduce_prefix_scan_gb300._abi import ak_linattn
    a = ak_linattn(100, 2, 0, 4, 64, 64, 2, 1.0, 0)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def test_linear_attention_refusals(L):
    from mapreduce_prefix_scan_gb300._abi import AK_ERR_INVALID_ARG as INV, AK_ERR_UNSUPPORTED as UNS, ak_heads
    H = lambda p=0x10000, t=256, h=64: ak_heads(p, t, h)
    R = ctypes.byref

    def fwd(a=None, q=H(), k=H(), v=H(), o=H(), ld=0x1000, off=0x2000, s0=None, s1=None):
        return L.ak_linear_attention(R(a or _linattn()), R(q), R(k), R(v), ld, off, s0, R(o), s1, None, 0, None, None)

    for bad in (dict(tokens=-1), dict(seqs=-1), dict(max_len=-1), dict(heads=0), dict(heads=70000), dict(dk=0), dict(dv=257),
                dict(dtype=99), dict(scale=float("nan")), dict(scale=float("inf")), dict(reserved=1), dict(tokens=1 << 40)):
        assert fwd(_linattn(**bad)) == INV, bad
    assert fwd(_linattn(dtype=1)) == UNS
    for bad in (dict(q=H(0)), dict(k=H(0x10001)), dict(v=H(t=-1)), dict(o=H(h=-64)), dict(o=H(h=0)), dict(o=H(t=64)),
                dict(o=H(t=255)), dict(ld=None), dict(ld=0x1001), dict(off=None), dict(off=0x2002), dict(s0=0x3001), dict(s1=0x3002)):
        assert fwd(**bad) == INV, bad
    assert L.ak_linear_attention(None, R(H()), R(H()), R(H()), 0x1000, 0x2000, None, R(H()), None, None, 0, None, None) == INV
    assert L.ak_linear_attention(R(_linattn()), None, R(H()), R(H()), 0x1000, 0x2000, None, R(H()), None, None, 0, None, None) == INV

    def bwd(a=None, do=H(), q=H(), dq=H(), dk=H(), dv=H(), ds=None, d0=None):
        return L.ak_linear_attention_backward(R(a or _linattn()), R(do), R(q), R(H()), R(H()), 0x1000, 0x2000, None, ds,
                                              R(dq), R(dk), R(dv), d0, None, 0, None, None)

    for bad in (dict(a=_linattn(heads=0)), dict(do=H(0)), dict(q=H(0)), dict(dq=H(h=0)), dict(dk=H(t=10)), dict(dv=H(0)),
                dict(ds=0x3001), dict(d0=0x3002), dict(ds=0x3000, d0=0x3000)):
        assert bwd(**bad) == INV, bad

    def step(a=None, state=0x4000, slots=0x5000, ns=5, o=H(), ld=0x1000):
        return L.ak_linear_attention_step(R(a or _linattn()), R(H()), R(H()), R(H()), ld, state, slots, ns, R(o), None, None)

    for bad in (dict(state=None), dict(state=0x4002), dict(slots=0x5001), dict(ns=-1), dict(o=H(h=0)), dict(ld=None),
                dict(a=_linattn(dk=300))):
        assert step(**bad) == INV, bad
    b = ctypes.c_size_t()
    assert L.ak_linear_attention_workspace_size(None, None, R(b)) == INV
    assert L.ak_linear_attention_workspace_size(R(_linattn()), None, None) == INV
    # nothing to do: no tokens and no state to pass on
    assert fwd(_linattn(tokens=0)) == 0 and step(_linattn(tokens=0)) == 0


def test_binding_refusals():
    torch = pytest.importorskip("torch")
    import mapreduce_prefix_scan_gb300 as ak
    x = torch.zeros(4, 2, 8)
    ld = torch.zeros(2)
    with pytest.raises(ValueError):
        ak.ak_linear_attention(x, x, x, ld)                       # not on a GPU
    with pytest.raises(ValueError):
        ak.ak_linear_attention(x.half(), x.half(), x.half(), ld)
    with pytest.raises(ValueError):
        ak.ak_linear_attention_step(x, x, x, ld, torch.zeros(4, 2, 8, 8))
    i = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError):
        ak.ak_batch_layout(i, i, torch.zeros(3, 2, dtype=torch.int32), i, block_size=16, max_tokens=3)
    with pytest.raises(ValueError):
        ak.ak_verify_drafts(torch.zeros(3, 2, 5), torch.zeros(3, 1, dtype=torch.int32), torch.zeros(3, 1), torch.zeros(3, 5))
