"""The gated recurrence, its gradients and its step against the recurrence in 64 bits.

Bounds, in units of 2^-24 of the sum of absolute values that a result adds up (`mass`): a token lies in a run of at
most 16 (bf16: 32), in a tile of 8 runs, in a cluster's step of at most 16 tiles. In a run each token costs its weights
and one rounding: 7 units in float32 (expf: 1 ulp, so 2 units; a sigmoid's exponential 4, its sum, reciprocal and
product), 11 in bf16 (exponential 4, sum, reciprocal 2, product, and the argument's rounding, as x e^-x <= 0.37). A run's
or tile's map costs an exponential (2 units, and 0.37 units for each of the at most 24 roundings of its logarithm) and two
roundings, less than 13 units. With tiles of 64 tokens at least: 16 * 7 (32 * 11) + (8 + tiles) * 13.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

import decoding_reference as ref
import mapreduce_prefix_scan_gb300 as ak

pytestmark = pytest.mark.gpu

U = 2.0**-24
HALF = {torch.float32: 2.0**-24, torch.bfloat16: 2.0**-8}


def units(tokens, dtype):
    return ((16 * 7 if dtype is torch.float32 else 32 * 11) + (8 + -(-tokens // 64)) * 13) * U


def _case(lens, channels, dtype, form, state=True, seed=0, before=0, after=0, spread=1.0):
    """Packed inputs with rows outside every sequence before and after."""
    g = torch.Generator().manual_seed(seed)
    t = before + sum(lens) + after
    gate = torch.randn(t, channels, generator=g)
    gate = -torch.exp(gate * 2 - 3) * spread if form == "decay" else gate * 2 + 1
    x, dh = torch.randn(t, channels, generator=g), torch.randn(t, channels, generator=g)
    s0 = torch.randn(len(lens), channels, generator=g) if state else None
    ds = torch.randn(len(lens), channels, generator=g) if state else None
    off = np.concatenate([[0], np.cumsum(lens)]) + before
    c = dict(x=x.to(dtype).cuda(), gate=gate.to(dtype).cuda(), dh=dh.to(dtype).cuda(),
             offsets=torch.tensor(off, dtype=torch.int32).cuda(), off=off.astype(int))
    c["s0"], c["ds"] = (None, None) if s0 is None else (s0.cuda(), ds.cuda())
    return c


def _np(t):
    return None if t is None else t.double().cpu().numpy()


def _close(got, want, bound, what):
    got = _np(got)
    bad = ~(np.abs(got - want) <= bound)
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:3].tolist(), got[bad][:3], want[bad][:3])


def _check_forward(c, form, h, sf):
    dtype = c["x"].dtype
    want, wsf, mass = ref.recurrence(_np(c["x"]), _np(c["gate"]), c["off"], _np(c["s0"]), form)
    e = units(len(want), dtype)
    _close(h, want, e * mass + HALF[dtype] * (np.abs(want) + e * mass) + 1e-37, "h")
    if sf is not None:
        sm = np.array([mass[c["off"][i + 1] - 1] if c["off"][i + 1] > c["off"][i] else np.zeros(want.shape[1]) for i in range(len(wsf))])
        _close(sf, wsf, e * sm + 1e-37, "state")


def _check_backward(c, form, h, grads):
    dtype = c["x"].dtype
    x = _np(c["x"])
    dx, dg, d0, gm, hm = ref.recurrence_gradients(_np(c["dh"]), x, _np(c["gate"]), c["off"], _np(c["s0"]), _np(c["ds"]), form)
    a, b = ref.weights(_np(c["gate"]), form)
    e = units(len(x), dtype)
    half = HALF[dtype]
    _close(grads[0], dx, b * (e * gm) + half * (np.abs(dx) + e * gm) + 1e-37, "dx")
    # h as it was stored: another half step of it, and its own error
    he = (2 * e + half) * hm
    ab = a if form == "decay" else a * b
    d = hm if form == "decay" else hm + np.abs(x)
    _close(grads[1], dg, ab * (gm * he + 2 * e * gm * d) + half * np.abs(dg) * (1 + 1e-2) + 1e-37, "dgate")
    if c["s0"] is not None:
        first = np.array([gm[c["off"][i]] * a[c["off"][i]] if c["off"][i + 1] > c["off"][i] else np.abs(d0[i]) for i in range(len(d0))])
        _close(grads[2], d0, e * first + 1e-37, "dstate")


LENS = {
    "one token": [1],
    "one": [300],
    "a tile exactly": [128],
    "packed": [70, 1, 0, 0, 130, 64, 3, 0],
    "single tokens": [1] * 150,
    "empty": [0, 0, 5],
    "many": [3, 0, 17, 1] * 60,
    "long": [2500, 1, 2200],
}


@pytest.mark.parametrize("form", ["decay", "gate"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("channels", [1, 64, 77, 136, 1000])
@pytest.mark.parametrize("name", LENS)
def test_forward_and_gradients(name, channels, dtype, form):
    if channels == 1000 and name == "long":
        channels = 320
    c = _case(LENS[name], channels, dtype, form, state=name not in ("one", "single tokens"), seed=len(name) + channels)
    h, sf = ak.ak_gated_recurrence(c["x"], c["gate"], form=form, offsets=c["offsets"], state=c["s0"], final_state=True)
    _check_forward(c, form, h, sf)
    grads = ak.ak_gated_recurrence_backward(c["dh"], c["x"], c["gate"], h, form=form, offsets=c["offsets"], state=c["s0"],
                                            dstate_out=c["ds"])
    _check_backward(c, form, h, grads)


@pytest.mark.parametrize("form", ["decay", "gate"])
@pytest.mark.parametrize("before,after", [(0, 9), (5, 0), (130, 200)])
def test_rows_outside_every_sequence(form, before, after):
    """They give zeros, whatever they hold."""
    c = _case([40, 90], 68, torch.float32, form, before=before, after=after)
    for t in ("x", "gate", "dh"):
        c[t][:before] = float("nan")
        c[t][before + 130:] = float("inf")
    h, sf = ak.ak_gated_recurrence(c["x"], c["gate"], form=form, offsets=c["offsets"], state=c["s0"], final_state=True)
    grads = ak.ak_gated_recurrence_backward(c["dh"], c["x"], c["gate"], h, form=form, offsets=c["offsets"], state=c["s0"], dstate_out=c["ds"])
    for t in (h, *grads[:2]):
        assert not t[:before].any() and not t[before + 130:].any()
    for t in ("x", "gate", "dh"):
        c[t][:before] = 0
        c[t][before + 130:] = 0
    _check_forward(c, form, h, sf)
    _check_backward(c, form, h, grads)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_views_of_a_packed_projection(dtype):
    """Rows with strides of their own, at any alignment; outputs into given views."""
    for channels, start in ((64, 0), (64, 1), (50, 3)):
        wide = torch.randn(210, 3 * channels + 5, device="cuda").to(dtype)
        x, gate, dh = (wide[:, start + i * channels: start + (i + 1) * channels] for i in range(3))
        off = torch.tensor([0, 110, 210], dtype=torch.int32, device="cuda")
        out = torch.full((210, channels + 3), 7.0, device="cuda", dtype=dtype)
        h, _ = ak.ak_gated_recurrence(x, gate, form="gate", offsets=off, out=out[:, 1:-2])
        plain, _ = ak.ak_gated_recurrence(x.contiguous(), gate.contiguous(), form="gate", offsets=off)
        assert torch.equal(h, plain) and (out[:, 0] == 7).all() and (out[:, -2:] == 7).all()
        a = ak.ak_gated_recurrence_backward(dh, x, gate, h, form="gate", offsets=off)
        b = ak.ak_gated_recurrence_backward(dh.contiguous(), x.contiguous(), gate.contiguous(), plain, form="gate", offsets=off)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_one_gate_for_all_tokens():
    """A gate row shared by stride 0; its gradient for each token."""
    c = _case([90, 33], 40, torch.float32, "decay")
    row = c["gate"][:1]
    shared, c["gate"] = row.expand(123, 40), row.repeat(123, 1)
    h, sf = ak.ak_gated_recurrence(c["x"], shared, offsets=c["offsets"], state=c["s0"], final_state=True)
    _check_forward(c, "decay", h, sf)
    _check_backward(c, "decay", h, ak.ak_gated_recurrence_backward(c["dh"], c["x"], shared, h, offsets=c["offsets"], state=c["s0"], dstate_out=c["ds"]))


@pytest.mark.parametrize("form", ["decay", "gate"])
def test_state_in_place(form):
    c = _case([40, 0, 300, 1], 100, torch.float32, form)
    want = ak.ak_gated_recurrence(c["x"], c["gate"], form=form, offsets=c["offsets"], state=c["s0"], final_state=True)
    s = c["s0"].clone()
    h, sf = ak.ak_gated_recurrence(c["x"], c["gate"], form=form, offsets=c["offsets"], state=s, state_out=s)
    assert sf is s and torch.equal(h, want[0]) and torch.equal(s, want[1]) and torch.equal(s[1], c["s0"][1])


def test_segments_agree_with_the_whole():
    """A sequence cut in two, its state handed on, and the gradient of the state handed back."""
    c = _case([700], 96, torch.float32, "gate")
    h, sf = ak.ak_gated_recurrence(c["x"], c["gate"], form="gate", state=c["s0"], final_state=True)
    h1, s1 = ak.ak_gated_recurrence(c["x"][:333], c["gate"][:333], form="gate", state=c["s0"], final_state=True)
    h2, s2 = ak.ak_gated_recurrence(c["x"][333:], c["gate"][333:], form="gate", state=s1, final_state=True)
    _check_forward(c, "gate", torch.cat([h1, h2]), s2)
    b2 = ak.ak_gated_recurrence_backward(c["dh"][333:], c["x"][333:], c["gate"][333:], h2, form="gate", state=s1, dstate_out=c["ds"])
    b1 = ak.ak_gated_recurrence_backward(c["dh"][:333], c["x"][:333], c["gate"][:333], h1, form="gate", state=c["s0"], dstate_out=b2[2])
    _check_backward(c, "gate", h, (torch.cat([b1[0], b2[0]]), torch.cat([b1[1], b2[1]]), b1[2]))


@pytest.mark.parametrize("form", ["decay", "gate"])
def test_nonfinite_values_stay_in_their_sequence_and_channel(form):
    c = _case([150, 150], 72, torch.float32, form, seed=3)
    clean = ak.ak_gated_recurrence(c["x"], c["gate"], form=form, offsets=c["offsets"], state=c["s0"], final_state=True)
    x, gate = c["x"].clone(), c["gate"].clone()
    x[60, 5] = float("nan")
    x[61, 6] = float("inf")
    gate[20, 7] = float("nan")
    h, sf = ak.ak_gated_recurrence(x, gate, form=form, offsets=c["offsets"], state=c["s0"], final_state=True)
    hit = torch.zeros_like(h, dtype=torch.bool)
    hit[60:150, 5] = hit[61:150, 6] = hit[20:150, 7] = True
    assert torch.equal(~torch.isfinite(h), hit)
    assert torch.equal(h[~hit], clean[0][~hit]) and torch.equal(sf[1], clean[1][1])
    # gradients: backwards in time
    dh = c["dh"].clone()
    dh[200, 3] = float("nan")
    same = dict(form=form, offsets=c["offsets"], state=c["s0"], dstate_out=c["ds"])
    want = ak.ak_gated_recurrence_backward(c["dh"], c["x"], c["gate"], clean[0], **same)
    got = ak.ak_gated_recurrence_backward(dh, c["x"], c["gate"], clean[0], **same)
    hit[:] = False
    hit[150:201, 3] = True
    assert torch.equal(~torch.isfinite(got[0]), hit) and torch.equal(got[0][~hit], want[0][~hit])
    assert torch.equal(got[1][~hit], want[1][~hit]) and torch.isnan(got[2][1, 3]) and torch.equal(got[2][0], want[2][0])


def test_gates_that_forget_and_that_keep():
    """-inf forgets (an infinity before it gives NaN, as 0 * inf does); logits of +-inf keep the state or take x alone."""
    x = torch.randn(70, 8, device="cuda")
    gate = torch.zeros(70, 8, device="cuda")
    gate[40] = -float("inf")
    h, _ = ak.ak_gated_recurrence(x, gate)
    torch.testing.assert_close(h[39], x[:40].sum(0), rtol=1e-4, atol=1e-4)
    assert torch.equal(h[40], x[40])
    logit = torch.full((70, 8), float("inf"), device="cuda")
    s0 = torch.randn(1, 8, device="cuda")
    h, sf = ak.ak_gated_recurrence(x, logit, form="gate", state=s0, final_state=True)
    assert torch.equal(h, s0.expand(70, 8)) and torch.equal(sf, s0)
    h, _ = ak.ak_gated_recurrence(x, -logit, form="gate", state=s0)
    assert torch.equal(h, x)


@pytest.mark.parametrize("form,gate", [("decay", -1e-4), ("decay", -1e-6), ("gate", 9.0)])
def test_long_memories_keep_their_precision(form, gate):
    """30000 tokens at one gate: in norm, against 64 bits. Factors a token at a time, each off by up to 2^-25 and all the
    same way, would be off by 3e-8 for every token remembered (1e4 of them: 3e-4). Here only a run's factors are rounded
    (up to 16 * 2^-25 = 4.8e-7 of what came before the run, and half of that of all that runs add), and a run's and a
    tile's two sums, whose roundings differ from state to state: sqrt(2 * (470 + 16)) * 2^-25 / 2 = 5e-7, in the mean.
    4.8e-7 + 2.4e-7 + 5e-7 = 1.22e-6."""
    t, ch = 30000, 64
    x = torch.randn(t, ch, device="cuda") + 0.5
    g = torch.full((t, ch), gate, device="cuda")
    h, sf = ak.ak_gated_recurrence(x, g, form=form, final_state=True)
    want, wsf, _ = ref.recurrence(_np(x), _np(g), [0, t], None, form)
    assert np.linalg.norm(_np(h) - want) <= 1.22e-6 * np.linalg.norm(want)
    assert np.linalg.norm(_np(sf) - wsf) <= 1.22e-6 * np.linalg.norm(wsf)


def test_gradients_against_differences():
    c = _case([9, 14], 8, torch.float32, "gate", seed=11)
    w, ws = c["dh"].double(), c["ds"].double()

    def loss(x, gate, s0):
        h, sf, _ = ref.recurrence(x, gate, c["off"], s0, "gate")
        return (h * _np(w)).sum() + (sf * _np(ws)).sum()

    h, _ = ak.ak_gated_recurrence(c["x"], c["gate"], form="gate", offsets=c["offsets"], state=c["s0"])
    grads = ak.ak_gated_recurrence_backward(c["dh"], c["x"], c["gate"], h, form="gate", offsets=c["offsets"], state=c["s0"], dstate_out=c["ds"])
    at = [_np(c[k]) for k in ("x", "gate", "s0")]
    for i, (name, g) in enumerate(zip(("x", "gate", "s0"), grads)):
        for j in ((0, 0), (1, 3), (at[i].shape[0] - 1, 7)):
            step = 1e-4
            up, down = [a.copy() for a in at], [a.copy() for a in at]
            up[i][j] += step
            down[i][j] -= step
            # a central difference is off by step^2 / 6 of the third derivative (of order 10) and 1e-15 / step
            assert abs((loss(*up) - loss(*down)) / (2 * step) - float(g[j])) <= 1e-5 * (1 + abs(float(g[j]))), name


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("form", ["decay", "gate"])
def test_recorded_gradients_are_those_of_the_backward_call(form, dtype):
    c = _case([70, 50], 48, dtype, form)
    x, gate, s0 = c["x"].requires_grad_(), c["gate"].requires_grad_(), c["s0"].requires_grad_()
    h, sf = ak.ak_gated_recurrence(x, gate, form=form, offsets=c["offsets"], state=s0, final_state=True)
    got = torch.autograd.grad([h, sf], [x, gate, s0], [c["dh"], c["ds"]])
    want = ak.ak_gated_recurrence_backward(c["dh"], x.detach(), gate.detach(), h.detach(), form=form, offsets=c["offsets"],
                                           state=s0.detach(), dstate_out=c["ds"])
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    # a sum's gradient has strides of zero; a shared gate row gets the sum
    row = gate.detach()[:1].clone().requires_grad_()
    h, _ = ak.ak_gated_recurrence(x, row.expand(120, 48), form=form, offsets=c["offsets"])
    h.sum().backward()
    _, dg, _ = ak.ak_gated_recurrence_backward(torch.ones_like(h), x.detach(), row.detach().expand(120, 48), h.detach(), form=form, offsets=c["offsets"])
    assert torch.equal(row.grad, dg.sum(0, keepdim=True))
    with pytest.raises(RuntimeError, match="gradient"):
        ak.ak_gated_recurrence(x, gate, form=form, out=torch.empty_like(h))[0].sum().backward()
    with pytest.raises(RuntimeError, match="gradient"):
        ak.ak_gated_recurrence_step(x, gate, torch.zeros(120, 48, device="cuda"), form=form).sum().backward()


@pytest.mark.parametrize("channels", [1, 7, 64, 130, 2560])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("form", ["decay", "gate"])
def test_step(form, dtype, channels):
    c = _case([1] * 9, channels, dtype, form)
    pool = torch.randn(12, channels, device="cuda")
    slots = torch.tensor([3, 11, 0, -1, 7, 12, 1, 5, 2147483647], dtype=torch.int32, device="cuda")
    was = pool.clone()
    h = ak.ak_gated_recurrence_step(c["x"], c["gate"], pool, form=form, slots=slots)
    a, b = ref.weights(_np(c["gate"]), form)
    for i, s in enumerate(slots.tolist()):
        if not 0 <= s < 12:
            assert not h[i].any()
            continue
        old, x = _np(was[s]), _np(c["x"][i])
        want, mass = a[i] * old + b[i] * x, a[i] * np.abs(old) + b[i] * np.abs(x)
        _close(pool[s], want, 8 * U * mass + 1e-37, "pool")
        _close(h[i], want, 9 * U * mass + HALF[dtype] * np.abs(want) + 1e-37, "h")
    rest = [i for i in range(12) if i not in slots.tolist()]
    assert torch.equal(pool[rest], was[rest])
    # steps follow one another as one sequence does
    s = torch.zeros(1, channels, device="cuda")
    rows = [ak.ak_gated_recurrence_step(c["x"][i: i + 1], c["gate"][i: i + 1], s, form=form) for i in range(9)]
    one = dict(c, s0=None, off=np.array([0, 9]))
    _check_forward(one, form, torch.cat(rows), s)


def test_calls_with_nothing_to_do():
    x = torch.zeros(0, 8, device="cuda")
    h, sf = ak.ak_gated_recurrence(x, x, offsets=torch.zeros(4, dtype=torch.int32, device="cuda"), final_state=True)
    assert h.shape == (0, 8) and sf.shape == (3, 8) and not sf.any()
    s0 = torch.randn(3, 8, device="cuda")
    _, sf = ak.ak_gated_recurrence(x, x, offsets=torch.zeros(4, dtype=torch.int32, device="cuda"), state=s0, final_state=True)
    assert torch.equal(sf, s0)
    y = torch.ones(5, 8, device="cuda")
    h, sf = ak.ak_gated_recurrence(y, -y, offsets=torch.zeros(1, dtype=torch.int32, device="cuda"), final_state=True)
    assert not h.any() and sf.shape == (0, 8)
    assert ak.ak_gated_recurrence_step(x, x, torch.zeros(2, 8, device="cuda")).shape == (0, 8)


def test_captured_and_replayed_beside_another_stream():
    """Equal bits on every replay, with two streams' calls in flight at once."""
    c = _case([500, 1, 800], 256, torch.bfloat16, "gate")
    call = lambda: ak.ak_gated_recurrence(c["x"], c["gate"], form="gate", offsets=c["offsets"], state=c["s0"], final_state=True)  # noqa: E731
    want = call()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        h, sf = call()
        grads = ak.ak_gated_recurrence_backward(c["dh"], c["x"], c["gate"], h, form="gate", offsets=c["offsets"], state=c["s0"])
    for _ in range(3):
        h.zero_()
        with torch.cuda.stream(side):
            other = call()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(h, want[0]) and torch.equal(sf, want[1]) and torch.equal(other[0], want[0])
    again = ak.ak_gated_recurrence_backward(c["dh"], c["x"], c["gate"], h, form="gate", offsets=c["offsets"], state=c["s0"])
    assert all(torch.equal(a, b) for a, b in zip(grads, again))


def test_rows_past_two_to_the_31():
    """Offsets of 64 bits: a strided view whose last row begins past 2^31 elements."""
    t, ch, stride = 40, 64, 60_000_000
    room = torch.empty(t * stride, dtype=torch.bfloat16, device="cuda")
    x, out = room.as_strided((t, ch), (stride, 1)), room.as_strided((t, ch), (stride, 1), 128)
    x.copy_(torch.randn(t, ch))
    gate = -torch.rand(t, ch, device="cuda").bfloat16()
    h, _ = ak.ak_gated_recurrence(x, gate, out=out)
    want, _ = ak.ak_gated_recurrence(x.contiguous(), gate)
    assert torch.equal(h, want)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_a_checked_call_ends_well(dtype):
    c = _case([700, 1, 900], 64, dtype, "gate")
    call = lambda o: ak.ak_gated_recurrence(c["x"], c["gate"], form="gate", offsets=c["offsets"], state=c["s0"], final_state=True, opts=o)  # noqa: E731
    h, sf = call(None)
    for limit in (0, 1):  # 1 ns: a wait lasts 0.1 s at least
        a, b = call(dict(check=True, wait_limit_ns=limit))
        assert torch.equal(a, h) and torch.equal(b, sf)
    back = lambda o: ak.ak_gated_recurrence_backward(c["dh"], c["x"], c["gate"], h, form="gate", offsets=c["offsets"], opts=o)  # noqa: E731
    assert all(torch.equal(a, b) for a, b in zip(back(None)[:2], back(dict(check=True))[:2]))
    s = c["s0"].clone()
    ak.ak_gated_recurrence_step(c["x"][:3], c["gate"][:3], s, opts=dict(check=True))


def test_a_wait_that_runs_out_is_reported():
    """A tile whose map is not sent: the blocks of its cluster give up after 0.1 s, and the next call is sound."""
    c = _case([1500, 1300], 64, torch.float32, "decay")
    call = lambda **o: ak.ak_gated_recurrence(c["x"], c["gate"], offsets=c["offsets"], state=c["s0"], final_state=True, opts=dict(check=True, **o))  # noqa: E731
    want = call()
    for tile in (0, 7):
        with pytest.raises(ak.AkError) as e:
            call(debug_skip_publish_tile=tile, wait_limit_ns=1)
        assert e.value.status == 6
        got = call()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_on_a_given_stream():
    c = _case([300, 200], 96, torch.bfloat16, "decay")
    want = ak.ak_gated_recurrence(c["x"], c["gate"], offsets=c["offsets"], state=c["s0"], final_state=True)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = ak.ak_gated_recurrence(c["x"], c["gate"], offsets=c["offsets"], state=c["s0"], final_state=True, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_equal_gates_in_bf16_calls():
    """States of bf16 calls at one gate: a run's 32 factors are exact to 2^-22 each (4 units of 2^-24, and one of
    rounding), and half of that of all that runs add: (32 + 16) * 5 * 2^-24 = 1.4e-5 if every one pushed as far as it may."""
    t, ch = 20000, 64
    x = (torch.randn(t, ch, device="cuda") + 0.5).bfloat16()
    for form, gate in (("decay", -1e-3), ("gate", 7.0)):
        g = torch.full((t, ch), gate, device="cuda").bfloat16()
        _, sf = ak.ak_gated_recurrence(x, g, form=form, final_state=True)
        _, wsf, _ = ref.recurrence(_np(x), _np(g), [0, t], None, form)
        assert np.linalg.norm(_np(sf) - wsf) <= 1.4e-5 * np.linalg.norm(wsf)


@pytest.mark.parametrize("form", ["decay", "gate"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("channels", [77, 320])
def test_in_place(channels, dtype, form):
    """Outputs in x's own memory."""
    c = _case([900, 0, 1, 1300], channels, dtype, form)
    want, ws = ak.ak_gated_recurrence(c["x"], c["gate"], form=form, offsets=c["offsets"], state=c["s0"], final_state=True)
    x = c["x"].clone()
    h, sf = ak.ak_gated_recurrence(x, c["gate"], form=form, offsets=c["offsets"], state=c["s0"], final_state=True, out=x)
    assert h is x and torch.equal(h, want) and torch.equal(sf, ws)
