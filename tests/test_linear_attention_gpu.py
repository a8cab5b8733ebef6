"""Linear attention with a decay for each head against its recurrence in 64 bits.

Bounds. float32: every output and state entry is a sum of at most
`tokens + dk` rounded products, each touched by a few more roundings (the
weights, the scale): |error| <= (tokens + dk + 16) 2^-24 M, M the sum of the
absolute values. bf16 (8 significant bits: a rounding is off by at most 2^-8
of the value): inputs are exact; the output rounds once (2^-8 |o|), each
weighted score and each entry of the state once where it enters a product
(2^-8 of the terms that went through scores and of those that went through the
state, M together), so |error| <= 2^-8 |o| + 2^-8 M + the float32 part.
States are float32 in either case: the float32 bound."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import mapreduce_prefix_scan_gb300 as ak
from sequence_reference import attention, attention_gradients

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def _dev(x, dtype=torch.float32):
    return None if x is None else torch.tensor(x, dtype=torch.float32, device="cuda").to(dtype)


def _inputs(seed, dtype, lens, h, dk, dv, state=True, ld=None):
    rng = np.random.default_rng(seed)
    t = sum(lens)
    r = lambda *s: torch.tensor(rng.normal(0, 1, s).astype(np.float32)).to(DT[dtype]).float().numpy()
    q, k, v, do = r(t, h, dk), r(t, h, dk), r(t, h, dv), r(t, h, dv)
    if ld is None:
        ld = -np.exp2(-8 * np.arange(1, h + 1) / h)
    n = len(lens)
    s0, ds = (rng.normal(0, 1, (2, n, h, dk, dv)).astype(np.float32) if state else (None, None))
    off = np.concatenate([[0], np.cumsum(lens)]).astype(np.int64)
    return q, k, v, do, np.asarray(ld, np.float32), off, s0, ds


def _bound(dtype, lens, dk, want, mass):
    f32 = (max(list(lens) + [1]) + dk + 16) * 2.0**-24 * mass
    return f32 if dtype == "f32" else 2.0**-8 * np.abs(want) + 2.0**-8 * mass + f32


def _close(got, want, tol, name):
    got = got.double().cpu().numpy()
    err = np.abs(got - want)
    assert got.shape == want.shape and np.isfinite(got).all(), name
    bad = err > tol + 1e-30
    assert not bad.any(), f"{name}: {bad.sum()} of {bad.size} off; worst ratio {np.max(err / (tol + 1e-30)):.3g} at {np.unravel_index(np.argmax(err / (tol + 1e-30)), err.shape)}"


def _off(off):
    return torch.tensor(off, dtype=torch.int32, device="cuda")


def _forward_case(dtype, lens, h, dk, dv, state=True, ld=None, scale=0.37, seed=0, **opts):
    q, k, v, do, ld, off, s0, ds = _inputs(seed, dtype, lens, h, dk, dv, state, ld)
    want, sf, mass = attention(q, k, v, ld, off, s0, scale)
    _, sa, _ = attention(np.abs(q), np.abs(k), np.abs(v), ld, off, None if s0 is None else np.abs(s0))
    d = DT[dtype]
    o, s1 = ak.ak_linear_attention(_dev(q, d), _dev(k, d), _dev(v, d), _dev(ld), offsets=_off(off), state=_dev(s0),
                                   scale=scale, final_state=True, opts=opts or None)
    _close(o, want, _bound(dtype, lens, dk, want, mass), "o")
    _close(s1, sf, _bound("f32", lens, dk, sf, sa), "state")
    return o, s1


def _mass_gradients(do, q, k, v, ld, off, s0, ds, scale):
    a = np.abs
    return attention_gradients(a(do), a(q), a(k), a(v), ld, off, None if s0 is None else a(s0),
                               None if ds is None else a(ds), abs(scale))


def _backward_case(dtype, lens, h, dk, dv, state=True, ld=None, scale=0.37, seed=1, **opts):
    q, k, v, do, ld, off, s0, ds = _inputs(seed, dtype, lens, h, dk, dv, state, ld)
    want = attention_gradients(do, q, k, v, ld, off, s0, ds, scale)
    mass = _mass_gradients(do, q, k, v, ld, off, s0, ds, scale)
    d = DT[dtype]
    got = ak.ak_linear_attention_backward(_dev(do, d), _dev(q, d), _dev(k, d), _dev(v, d), _dev(ld), offsets=_off(off),
                                          state=_dev(s0), dstate_out=_dev(ds), scale=scale, opts=opts or None)
    for i, name in enumerate(("dq", "dk", "dv")):
        _close(got[i], want[i], _bound(dtype, lens, max(dk, dv), want[i], mass[i]), name)
    if state:
        _close(got[3], want[3], _bound("f32", lens, max(dk, dv), want[3], mass[3]), "dstate")
    else:
        assert got[3] is None


SHAPES = [
    ([1], 1, 64, 64), ([5], 3, 128, 128), ([63], 2, 64, 64), ([64], 2, 128, 128), ([65], 1, 64, 64), ([129], 2, 128, 128),
    ([200], 1, 128, 128), ([0, 3, 0, 0, 70, 1, 0], 2, 64, 64), ([130, 1, 0, 127, 128, 2], 2, 128, 128),
    ([17, 40], 3, 1, 1), ([33], 2, 80, 48), ([50, 9], 1, 5, 3), ([20], 1, 256, 256), ([40, 41], 2, 128, 64), ([31], 2, 33, 100),
]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("lens,h,dk,dv", SHAPES)
def test_forward(dtype, lens, h, dk, dv):
    _forward_case(dtype, lens, h, dk, dv)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("lens,h,dk,dv", SHAPES)
def test_backward(dtype, lens, h, dk, dv):
    _backward_case(dtype, lens, h, dk, dv)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("windows", [1, 2, 5, 100])
@pytest.mark.parametrize("state", [False, True])
def test_windows_of_the_token_axis(dtype, windows, state):
    """Sequences that end on, before and after the windows' ends, and one that spans many windows."""
    lens = [64, 1, 63, 0, 300, 128, 0, 7]
    _forward_case(dtype, lens, 2, 64, 64, state=state, target_blocks=windows)
    _backward_case(dtype, lens, 2, 64, 64, state=state, target_blocks=windows)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("windows", [1, 3])
def test_decays_from_none_to_complete(dtype, windows):
    """No decay, slow, fast, faster than float32's range over a chunk, and no memory at all."""
    ld = [0.0, -1e-5, -0.3, -3.0, -60.0, -200.0, -np.inf]
    _forward_case(dtype, [150, 60], 7, 64, 64, ld=ld, target_blocks=windows)
    _backward_case(dtype, [150, 60], 7, 64, 64, ld=ld, target_blocks=windows)


def test_slow_decay_keeps_its_precision():
    """A memory of 10000 tokens, all terms of one sign: a factor off by 2^-24 would show as 2^-24 of every
    token's age. Sums of 3000 terms against the float32 bound."""
    t = 3000
    for dtype in ("f32", "bf16"):
        ones = torch.ones(t, 1, 64, device="cuda", dtype=DT[dtype])
        ld = np.array([-1e-4], np.float32)
        _, s = ak.ak_linear_attention(ones, ones, ones, _dev(ld), final_state=True)
        g = np.exp(np.float64(ld[0]))
        want = (1 - g**t) / (1 - g)
        # 64 additions in a chunk of exact ones times weights good to 2^-23, then t / 64 rounded steps
        assert abs(float(s[0, 0, 3, 5]) - want) <= (t / 16 + 16) * 2.0**-24 * want
        assert float(s.max()) - float(s.min()) <= 2.0**-20 * want


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("dim", [64, 80, 128])
def test_views_of_a_packed_projection_and_heads_first(dtype, dim):
    lens, h = [70, 3, 90], 3
    q, k, v, do, ld, off, s0, ds = _inputs(3, dtype, lens, h, dim, dim)
    d, t = DT[dtype], sum(lens)
    qkv = torch.stack([_dev(x, d) for x in (q, k, v)], 1)            # [t, 3, h, dim]
    want, sf, mass = attention(q, k, v, ld, off, s0)
    out = torch.full((h, t, dim), 9.0, device="cuda", dtype=d)       # heads first
    o, _ = ak.ak_linear_attention(qkv[:, 0], qkv[:, 1], qkv[:, 2], _dev(ld), offsets=_off(off), state=_dev(s0),
                                  out=out.transpose(0, 1))
    _close(o, want, _bound(dtype, lens, dim, want, mass), "o")
    # rows at offsets that 16-byte loads cannot take
    pad = torch.zeros(t, h, dim + 3, device="cuda", dtype=d)
    odd = [pad.clone()[:, :, 1:1 + dim].copy_(_dev(x, d)) for x in (q, k, v)]
    o, s1 = ak.ak_linear_attention(*odd, _dev(ld), offsets=_off(off), state=_dev(s0), final_state=True)
    _close(o, want, _bound(dtype, lens, dim, want, mass), "o")
    g = ak.ak_linear_attention_backward(_dev(do, d), qkv[:, 0], qkv[:, 1], qkv[:, 2], _dev(ld), offsets=_off(off),
                                        state=_dev(s0), dstate_out=_dev(ds))
    want = attention_gradients(do, q, k, v, ld, off, s0, ds)
    mass = _mass_gradients(do, q, k, v, ld, off, s0, ds, 1.0)
    for i in range(3):
        _close(g[i], want[i], _bound(dtype, lens, dim, want[i], mass[i]), "gradient %d" % i)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_a_head_shared_by_all(dtype):
    """k of one head read by all (head stride 0)."""
    q, k, v, _, ld, off, s0, _ = _inputs(4, dtype, [100], 4, 64, 64)
    k = np.broadcast_to(k[:, :1], k.shape)
    want, _, mass = attention(q, k, v, ld, off, s0)
    kk = _dev(np.ascontiguousarray(k[:, :1]), DT[dtype]).expand(100, 4, 64)
    o, _ = ak.ak_linear_attention(_dev(q, DT[dtype]), kk, _dev(v, DT[dtype]), _dev(ld), offsets=_off(off), state=_dev(s0))
    _close(o, want, _bound(dtype, [100], 64, want, mass), "o")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("windows", [1, 4])
def test_tokens_outside_every_sequence_are_zero_and_do_not_leak(dtype, windows):
    q, k, v, do, ld, off, s0, ds = _inputs(5, dtype, [40, 90], 2, 64, 64)
    d = DT[dtype]
    t, lo = 260, 37  # tokens before the first and after the last sequence hold NaN
    grow = lambda x: torch.full((t,) + x.shape[1:], float("nan"), device="cuda", dtype=d).index_copy_(
        0, torch.arange(lo, lo + 130, device="cuda"), _dev(x, d))
    off2 = off + lo
    o, s1 = ak.ak_linear_attention(grow(q), grow(k), grow(v), _dev(ld), offsets=_off(off2), state=_dev(s0),
                                   final_state=True, opts=dict(target_blocks=windows))
    want, sf, mass = attention(q, k, v, ld, off, s0)
    assert (o[:lo] == 0).all() and (o[lo + 130:] == 0).all()
    _close(o[lo:lo + 130], want, _bound(dtype, [90], 64, want, mass), "o")
    assert torch.isfinite(s1).all()
    g = ak.ak_linear_attention_backward(grow(do), grow(q), grow(k), grow(v), _dev(ld), offsets=_off(off2),
                                        state=_dev(s0), dstate_out=_dev(ds), opts=dict(target_blocks=windows))
    want = attention_gradients(do, q, k, v, ld, off, s0, ds)
    mass = _mass_gradients(do, q, k, v, ld, off, s0, ds, 1.0)
    for i in range(3):
        assert (g[i][:lo] == 0).all() and (g[i][lo + 130:] == 0).all()
        _close(g[i][lo:lo + 130], want[i], _bound(dtype, [90], 64, want[i], mass[i]), "gradient %d" % i)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_a_nan_stays_in_its_sequence_and_head(dtype):
    q, k, v, _, ld, off, s0, _ = _inputs(6, dtype, [70, 50, 60], 2, 64, 64)
    v[75, 1, 3] = np.nan
    k[76, 1, 3] = np.inf
    o, s1 = ak.ak_linear_attention(_dev(q, DT[dtype]), _dev(k, DT[dtype]), _dev(v, DT[dtype]), _dev(ld),
                                   offsets=_off(off), state=_dev(s0), final_state=True)
    assert torch.isfinite(o[:, 0]).all() and torch.isfinite(o[:70]).all() and torch.isfinite(o[120:]).all()
    assert torch.isnan(o[76:120, 1, 3]).all()
    assert torch.isfinite(s1[0]).all() and torch.isfinite(s1[2]).all() and torch.isnan(s1[1, 1, :, 3]).any()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_equal_calls_give_equal_bits_and_a_split_sequence_continues(dtype):
    a = _forward_case(dtype, [200, 90], 2, 64, 64)
    b = _forward_case(dtype, [200, 90], 2, 64, 64)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    q, k, v, _, ld, off, s0, _ = _inputs(0, dtype, [300], 2, 128, 128)
    d = DT[dtype]
    q, k, v, ld = _dev(q, d), _dev(k, d), _dev(v, d), _dev(ld)
    s = _dev(s0)
    whole, s_whole = ak.ak_linear_attention(q, k, v, ld, state=s, final_state=True)
    parts = []
    for x, y in ((0, 1), (1, 130), (130, 300)):
        o, _ = ak.ak_linear_attention(q[x:y], k[x:y], v[x:y], ld, state=s, state_out=s)  # in place
        parts.append(o)
    want, sf, mass = attention(*[x.double().cpu().numpy() for x in (q, k, v)], ld.cpu().numpy(), off, s0)
    _close(torch.cat(parts), want, _bound(dtype, [300], 128, want, mass), "o")
    _, sa, _ = attention(*[x.double().abs().cpu().numpy() for x in (q, k, v)], ld.cpu().numpy(), off, np.abs(s0))
    _close(s, sf, _bound("f32", [300], 128, sf, sa), "state")


@pytest.mark.parametrize("dtype,dim", [("f32", 64), ("bf16", 64), ("bf16", 128), ("bf16", 80)])
@pytest.mark.parametrize("windows", [1, 7, 0])
def test_states_in_place(dtype, dim, windows):
    """state_out may be state_in whatever the windows: the bits of a call with two buffers."""
    q, k, v, _, ld, off, s0, _ = _inputs(11, dtype, [200, 0, 64, 500, 3], 2, dim, dim)
    a = [_dev(x, DT[dtype]) for x in (q, k, v)] + [_dev(ld)]
    opts = dict(target_blocks=windows)
    o, s1 = ak.ak_linear_attention(*a, offsets=_off(off), state=_dev(s0), final_state=True, opts=opts)
    s = _dev(s0)
    for _ in range(3):
        s.copy_(_dev(s0))
        o2, _ = ak.ak_linear_attention(*a, offsets=_off(off), state=s, state_out=s, opts=opts)
        assert torch.equal(o, o2) and torch.equal(s, s1)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_many_even_sequences(dtype):
    """A block for each sequence (max_len says that none is long)."""
    lens = [3, 1, 5, 0, 4, 70, 2, 1] * 6
    q, k, v, do, ld, off, s0, ds = _inputs(12, dtype, lens, 2, 64, 64)
    d = DT[dtype]
    a = [_dev(x, d) for x in (q, k, v)] + [_dev(ld)]
    o, s1 = ak.ak_linear_attention(*a, offsets=_off(off), state=_dev(s0), final_state=True, max_len=70)
    want, sf, mass = attention(q, k, v, ld, off, s0)
    _, sa, _ = attention(np.abs(q), np.abs(k), np.abs(v), ld, off, np.abs(s0))
    _close(o, want, _bound(dtype, lens, 64, want, mass), "o")
    _close(s1, sf, _bound("f32", lens, 64, sf, sa), "state")
    g = ak.ak_linear_attention_backward(_dev(do, d), *a, offsets=_off(off), state=_dev(s0), dstate_out=_dev(ds), max_len=70)
    want = attention_gradients(do, q, k, v, ld, off, s0, ds)
    mass = _mass_gradients(do, q, k, v, ld, off, s0, ds, 1.0)
    for i in range(3):
        _close(g[i], want[i], _bound(dtype, lens, 64, want[i], mass[i]), "gradient %d" % i)
    _close(g[3], want[3], _bound("f32", lens, 64, want[3], mass[3]), "dstate")


def test_no_tokens():
    z = torch.empty(0, 2, 64, device="cuda")
    ld = _dev(np.array([-0.1, -0.2]))
    s = torch.randn(3, 2, 64, 64, device="cuda")
    o, s1 = ak.ak_linear_attention(z, z, z, ld, offsets=_off([0, 0, 0, 0]), state=s, final_state=True)
    assert o.shape == (0, 2, 64) and torch.equal(s, s1)
    g = ak.ak_linear_attention_backward(z, z, z, z, ld, offsets=_off([0, 0, 0, 0]), state=s, dstate_out=s)
    assert torch.equal(g[3], s)


def test_differences():
    """The operator is linear in each input by itself, so a central difference of any width is exact up to the
    rounding of the two losses it subtracts (their terms' absolute sum times 2^-20)."""
    lens, h, d = [70, 0, 45], 2, 64
    q, k, v, do, ld, off, s0, ds = _inputs(7, "f32", lens, h, d, d)
    x = dict(q=_dev(q), k=_dev(k), v=_dev(v), s=_dev(s0))
    rest = (_dev(ld),)
    g = dict(zip(("q", "k", "v", "s"), ak.ak_linear_attention_backward(
        _dev(do), x["q"], x["k"], x["v"], *rest, offsets=_off(off), state=x["s"], dstate_out=_dev(ds), scale=0.3)))

    def loss(**y):
        o, s = ak.ak_linear_attention(y["q"], y["k"], y["v"], *rest, offsets=_off(off), state=y["s"], scale=0.3,
                                      final_state=True)
        a, b = o.double() * _dev(do).double(), s.double() * _dev(ds).double()
        return float(a.sum() + b.sum()), float(a.abs().sum() + b.abs().sum())

    torch.manual_seed(0)
    for name in x:
        step = torch.randn_like(x[name])
        up, m1 = loss(**{**x, name: x[name] + step})
        down, m2 = loss(**{**x, name: x[name] - step})
        want = float((g[name].double() * step.double()).sum())
        assert abs((up - down) / 2 - want) <= 2.0**-20 * (m1 + m2) + 2.0**-20 * float((g[name].double() * step.double()).abs().sum()), name


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("b,h,dk,dv", [(1, 1, 64, 64), (1, 16, 128, 128), (5, 3, 80, 48), (70, 8, 128, 128), (4, 2, 3, 5),
                                       (3, 2, 256, 256), (2, 2, 17, 100), (400, 1, 32, 40)])
def test_step(dtype, b, h, dk, dv):
    rng = np.random.default_rng(b)
    q, k, v, _, ld, _, _, _ = _inputs(b, dtype, [b], h, dk, dv, state=False)
    pool = rng.normal(0, 1, (b + 3, h, dk, dv)).astype(np.float32)
    slots = rng.permutation(b + 3)[:b]
    if b > 2:
        slots[1], slots[2] = -1, b + 3  # padding
    d = DT[dtype]
    s = _dev(pool)
    qkv = torch.cat([_dev(x, d) for x in (q, k, v)], 2)
    o = ak.ak_linear_attention_step(qkv[..., :dk], qkv[..., dk:2 * dk], qkv[..., 2 * dk:], _dev(ld), s,
                                    slots=torch.tensor(slots, dtype=torch.int32, device="cuda"), scale=0.7)
    want, mass, new = np.zeros((b, h, dv)), np.zeros((b, h, dv)), pool.astype(np.float64)
    for i, x in enumerate(slots):
        if 0 <= x < b + 3:
            new[x] = np.exp(ld.astype(np.float64))[:, None, None] * new[x] + k[i][:, :, None].astype(np.float64) * v[i][:, None, :]
            want[i] = 0.7 * np.einsum("hi,hij->hj", q[i], new[x])
            mass[i] = 0.7 * np.einsum("hi,hij->hj", np.abs(q[i]), np.abs(new[x]))
    out_round = 2.0**-8 * np.abs(want) if dtype == "bf16" else 0
    _close(o, want, out_round + (dk + 16) * 2.0**-24 * mass, "o")
    _close(s, new, 4 * 2.0**-24 * (np.abs(new) + np.abs(pool)), "state")


def test_step_follows_the_prompt_form():
    q, k, v, _, ld, off, s0, _ = _inputs(8, "f32", [30], 2, 64, 64)
    a = [_dev(x) for x in (q, k, v)]
    _, mid = ak.ak_linear_attention(*[x[:20] for x in a], _dev(ld), state=_dev(s0), final_state=True)
    outs = [ak.ak_linear_attention_step(a[0][i:i + 1], a[1][i:i + 1], a[2][i:i + 1], _dev(ld), mid) for i in range(20, 30)]
    want, sf, mass = attention(q, k, v, ld, off, s0)
    _close(torch.cat(outs), want[20:], _bound("f32", [30], 64, want, mass)[20:], "o")


@pytest.mark.parametrize("dtype,dim", [("f32", 64), ("bf16", 64)])
def test_rows_further_apart_than_32_bits(dtype, dim):
    """Token strides that put the last rows beyond element 2^31, inputs, outputs and gradients."""
    t, step, h = 130, 17_000_000, 2
    q, k, v, do, ld, off, _, _ = _inputs(13, dtype, [t], h, dim, dim, state=False)
    d = DT[dtype]
    buf = torch.empty(t * step, dtype=d, device="cuda")

    def put(x, at):
        y = torch.as_strided(buf, (t, h, dim), (step, dim, 1), at)
        return y.copy_(_dev(x, d)) if x is not None else y

    w = h * dim
    a = [put(x, i * w) for i, x in enumerate((q, k, v))]
    o, _ = ak.ak_linear_attention(*a, _dev(ld), out=put(None, 3 * w), scale=0.4)
    want, _, mass = attention(q, k, v, ld, off, None, 0.4)
    _close(o, want, _bound(dtype, [t], dim, want, mass), "o")
    g = ak.ak_linear_attention_backward(put(do, 4 * w), *a, _dev(ld), dq=put(None, 5 * w), dk=put(None, 6 * w),
                                        dv=put(None, 7 * w), scale=0.4)
    want = attention_gradients(do, q, k, v, ld, off, None, None, 0.4)
    mass = _mass_gradients(do, q, k, v, ld, off, None, None, 0.4)
    for i in range(3):
        _close(g[i], want[i], _bound(dtype, [t], dim, want[i], mass[i]), "gradient %d" % i)


def test_step_in_a_pool_of_more_than_2_31_values():
    h, dim, slots = 32, 128, 4200
    pool = torch.empty(slots, h, dim, dim, device="cuda")
    rng = np.random.default_rng(14)
    q, k, v, _, ld, _, _, _ = _inputs(14, "f32", [2], h, dim, dim, state=False)
    s = rng.normal(0, 1, (2, h, dim, dim)).astype(np.float32)
    at = [slots - 1, 3]
    pool[at] = _dev(s)
    o = ak.ak_linear_attention_step(_dev(q), _dev(k), _dev(v), _dev(ld), pool,
                                    slots=torch.tensor(at, dtype=torch.int32, device="cuda"))
    new = np.exp(ld.astype(np.float64))[None, :, None, None] * s + k[..., :, None].astype(np.float64) * v[..., None, :]
    _close(pool[at], new, 4 * 2.0**-24 * (np.abs(new) + np.abs(s)), "state")
    _close(o, np.einsum("bhi,bhij->bhj", q, new), (dim + 16) * 2.0**-24 * np.einsum("bhi,bhij->bhj", np.abs(q), np.abs(new)), "o")


def test_other_stream_graph_and_workspace():
    q, k, v, _, ld, off, s0, _ = _inputs(9, "bf16", [400], 2, 64, 64)
    d = torch.bfloat16
    a = [_dev(x, d) for x in (q, k, v)]
    size = ak.ak_linear_attention_workspace_size(400, 2, 64, 64)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    base, _ = ak.ak_linear_attention(*a, _dev(ld), workspace=ws)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    o, _ = ak.ak_linear_attention(*a, _dev(ld), stream=side)
    side.synchronize()
    assert torch.equal(o, base)
    ldd = _dev(ld)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        o, _ = ak.ak_linear_attention(*a, ldd, workspace=ws)
    a[2].mul_(2)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, base * 2)  # a power of two passes through every rounding
    if size > 256:
        with pytest.raises(ValueError):
            ak.ak_linear_attention(*a, _dev(ld), workspace=ws[:size - 256])
