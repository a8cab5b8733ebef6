"""The gated linear recurrence over torch tensors: packed prompts, gradients,
single tokens.

These functions only marshal arguments; include/ak.h states the mathematics
and the rules of every argument. Tensors are ``[tokens, channels]`` (any token
stride, the channels contiguous), states ``[sequences, channels]`` float32.
"""
from __future__ import annotations

import torch

from . import _abi
from . import sequence as _s
from ._abi import FORMS, ak_recurrence, ak_rows


def _rows(t, shape, dtype, name, on):
    s = t.stride()
    if not (t.dtype is dtype and t.shape == shape and t.get_device() == on and (s[1] == 1 or shape[1] == 1)):
        raise ValueError(f"{name}: a {list(shape)} {dtype} tensor on x's CUDA device with contiguous channels is needed, "
                         f"got {list(t.shape)} {t.dtype} with strides {list(s)} on {t.device}")
    return ak_rows(t.data_ptr(), s[0])


def _state(t, shape, name, on):
    if t is None:
        return None
    if not (t.get_device() == on and t.dtype is torch.float32 and t.shape == shape and t.is_contiguous()):
        raise ValueError(f"{name}: a contiguous {list(shape)} float32 tensor on x's CUDA device is needed, "
                         f"got {list(t.shape)} {t.dtype} on {t.device}")
    return t.data_ptr()


def _geometry(x, offsets, form):
    if x.dim() != 2:
        raise ValueError("x and gate are [tokens, channels] tensors")
    kind, on = _s._FLOAT.get(x.dtype), x.get_device()
    if kind is None or on < 0:
        raise ValueError("x and gate are float32 or bfloat16 CUDA tensors")
    if form not in FORMS:
        raise ValueError(f"form is one of {list(FORMS)}")
    n, off = 1, None
    if offsets is not None:
        n = offsets.numel() - 1
        if n < 0:
            raise ValueError("offsets: at least one value is needed")
        off = _s._flat(offsets, torch.int32, n + 1, "offsets", on)
    t, c = x.shape
    return ak_recurrence(t, n, c, kind, FORMS[form]), (n, c), off, on


def _tracked(x, gate, state):
    return (x.requires_grad or gate.requires_grad or (state is not None and state.requires_grad)) and torch.is_grad_enabled()


class _Recurrence(torch.autograd.Function):
    """ak_gated_recurrence with its gradients in the graph."""

    @staticmethod
    def forward(ctx, x, gate, state, offsets, form, final_state, opts):
        h, state_out = ak_gated_recurrence(x, gate, form=form, offsets=offsets, state=state, final_state=final_state, opts=opts)
        ctx.save_for_backward(x, gate, state, offsets, h)
        ctx.rest = dict(form=form, opts=opts)
        ctx.set_materialize_grads(False)
        return h, state_out

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dh, dstate_out):
        x, gate, state, offsets, h = ctx.saved_tensors
        if dh is None:
            dh = torch.zeros_like(h)
        elif not _s._dense_rows(dh):
            dh = dh.contiguous()
        dstate_out = None if dstate_out is None else dstate_out.contiguous()
        dx, dgate, dstate = ak_gated_recurrence_backward(dh, x, gate, h, state=state, offsets=offsets, dstate_out=dstate_out,
                                                         **ctx.rest)
        return dx, dgate, dstate, None, None, None, None


def ak_gated_recurrence(x: torch.Tensor, gate: torch.Tensor, *, form: str = "decay", offsets: torch.Tensor | None = None,
                        state: torch.Tensor | None = None, out: torch.Tensor | None = None,
                        state_out: torch.Tensor | None = None, final_state: bool = False, opts=None, stream=None):
    """``h_t = a_t h_{t-1} + b_t x_t`` for every channel over packed sequences
    (``offsets`` int32, None: one sequence), from ``state`` [sequences, channels]
    float32 or zero. ``form="decay"``: a = exp(gate), b = 1; ``"gate"``: a =
    sigmoid(gate), b = 1 - a. Returns ``(h, state_out)``, the latter None unless
    given or asked for by ``final_state``. Gradients of x, gate and ``state`` are
    recorded as usual, of results that the call allocates on the current stream."""
    if _tracked(x, gate, state):
        if out is None and state_out is None and stream is None:
            return _Recurrence.apply(x, gate, state, offsets, form, final_state, opts)
        with torch.no_grad():
            results = ak_gated_recurrence(x, gate, form=form, offsets=offsets, state=state, out=out, state_out=state_out,
                                          final_state=final_state, opts=opts, stream=stream)
        return _s._Untracked.apply(results, "ak_gated_recurrence into given memory or on a given stream is not recorded: "
                                   "no gradient", x, gate, state)
    a, ss, off, on = _geometry(x, offsets, form)
    given = out, state_out
    if out is None:
        out = _s._empty(x.shape, x.dtype, x.device, stream)
    if state_out is None and final_state:
        state_out = _s._empty(ss, torch.float32, x.device, stream)
    shape, dt = x.shape, x.dtype
    rx, rg, ro = _rows(x, shape, dt, "x", on), _rows(gate, shape, dt, "gate", on), _rows(out, shape, dt, "out", on)
    _s._check(_abi.load().ak_gated_recurrence(a, rx, rg, off, _state(state, ss, "state", on), ro,
                                              _state(state_out, ss, "state_out", on), _s._opts(opts),
                                              _s._stream_of(stream, x)), "ak_gated_recurrence")
    _s._written(*given)
    return out, state_out


def ak_gated_recurrence_backward(dh: torch.Tensor, x: torch.Tensor, gate: torch.Tensor, h: torch.Tensor, *,
                                 form: str = "decay", offsets: torch.Tensor | None = None,
                                 state: torch.Tensor | None = None, dstate_out: torch.Tensor | None = None,
                                 dx: torch.Tensor | None = None, dgate: torch.Tensor | None = None,
                                 dstate: torch.Tensor | None = None, opts=None, stream=None):
    """Gradients of ak_gated_recurrence with respect to x, gate and the initial
    state, from the output ``h``, its gradient ``dh`` and the final state's
    ``dstate_out`` (or None). Returns ``(dx, dgate, dstate)``; ``dstate`` is None
    where the forward call had no ``state`` and none is given."""
    a, ss, off, on = _geometry(x, offsets, form)
    given = dx, dgate, dstate
    dx = _s._empty(x.shape, x.dtype, x.device, stream) if dx is None else dx
    dgate = _s._empty(x.shape, x.dtype, x.device, stream) if dgate is None else dgate
    if dstate is None and state is not None:
        dstate = _s._empty(ss, torch.float32, x.device, stream)
    shape, dt = x.shape, x.dtype
    rd, rx, rg = _rows(dh, shape, dt, "dh", on), _rows(x, shape, dt, "x", on), _rows(gate, shape, dt, "gate", on)
    rh, rdx, rdg = _rows(h, shape, dt, "h", on), _rows(dx, shape, dt, "dx", on), _rows(dgate, shape, dt, "dgate", on)
    _s._check(_abi.load().ak_gated_recurrence_backward(
        a, rd, rx, rg, rh, off, _state(state, ss, "state", on), _state(dstate_out, ss, "dstate_out", on), rdx, rdg,
        _state(dstate, ss, "dstate", on), _s._opts(opts), _s._stream_of(stream, x)), "ak_gated_recurrence_backward")
    _s._written(*given)
    return dx, dgate, dstate


def ak_gated_recurrence_step(x: torch.Tensor, gate: torch.Tensor, state: torch.Tensor, *, form: str = "decay",
                             slots: torch.Tensor | None = None, out: torch.Tensor | None = None, opts=None,
                             stream=None) -> torch.Tensor:
    """One token of each of ``x.shape[0]`` requests: updates the rows
    ``state[slots]`` ([slots, channels] float32; ``slots`` int32, None: request b
    uses state[b]) in place and returns the outputs. Slots outside the pool
    mark padding and give zeros. It has no gradient."""
    if _tracked(x, gate, state):
        with torch.no_grad():
            out = ak_gated_recurrence_step(x, gate, state, form=form, slots=slots, out=out, opts=opts, stream=stream)
        return _s._Untracked.apply((out,), "ak_gated_recurrence_step has no gradient", x, gate, state)[0]
    a, (_, c), _, on = _geometry(x, None, form)
    given = out
    if out is None:
        out = _s._empty(x.shape, x.dtype, x.device, stream)
    shape, dt = x.shape, x.dtype
    rx, rg, ro = _rows(x, shape, dt, "x", on), _rows(gate, shape, dt, "gate", on), _rows(out, shape, dt, "out", on)
    pool = state.shape[0]
    sp = _state(state, (pool, c), "state", on)
    at = None if slots is None else _s._flat(slots, torch.int32, x.shape[0], "slots", on)
    if slots is None and pool < x.shape[0]:
        raise ValueError("state: a row for each request is needed")
    _s._check(_abi.load().ak_gated_recurrence_step(a, rx, rg, sp, at, pool, ro, _s._opts(opts), _s._stream_of(stream, x)),
              "ak_gated_recurrence_step")
    _s._written(state, given)
    return out
