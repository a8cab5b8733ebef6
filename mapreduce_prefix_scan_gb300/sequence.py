"""The sequence operators over torch tensors: the layout of a batch from its
request lengths, the verification of drafted tokens, and linear attention
with a decay for each head (packed prompts, gradients, single tokens).

Like the rest of the binding these functions only marshal arguments; include/ak.h
states the mathematics and the rules of every argument. Tensors here are
plain row-major: ``[tokens, heads, dim]`` (any token and head stride, the last
dimension contiguous) and states ``[sequences, heads, dk, dv]``.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple

import torch

from . import _abi
from ._abi import DTYPES, ak_heads, ak_linattn

_FLOAT = {torch.float32: DTYPES["f32"], torch.bfloat16: DTYPES["bf16"]}


class BatchLayout(NamedTuple):
    """What ak_batch_layout fills in; ``counts`` holds the batch's tokens and the free blocks it takes."""
    offsets: torch.Tensor
    slots: torch.Tensor
    positions: torch.Tensor
    requests: torch.Tensor
    counts: torch.Tensor


# the handle alone: torch.cuda.current_stream() builds an object around it, which takes longer than a call here
_current = getattr(torch._C, "_cuda_getCurrentRawStream", None)


_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _stream_of(stream, t) -> int:
    """The stream of a call on t's device, which has to be the current one: the kernels run there."""
    on = t.get_device()
    if _device() != on:
        raise ValueError(f"the call's tensors are on device {on}, the current CUDA device is {_device()}")
    if stream is None:
        if _current is not None:
            return _current(on)
        return torch.cuda.current_stream(t.device).cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _empty(size, dtype, device, stream):
    """Memory for a call on `stream`: from that stream's own pool, so that nothing queued elsewhere still uses it."""
    if stream is None:
        return torch.empty(size, dtype=dtype, device=device)
    with torch.cuda.stream(stream if hasattr(stream, "cuda_stream") else torch.cuda.ExternalStream(int(stream), device)):
        return torch.empty(size, dtype=dtype, device=device)


def _opts(opts):
    if opts is None:
        return None
    from . import make_opts
    return ctypes.byref(make_opts(**opts) if isinstance(opts, dict) else opts)


def _check(status: int, where: str) -> None:
    if status:
        from . import AkError
        raise AkError(status, where)


def _need(cond, message):
    if not cond:
        raise ValueError(message)


def _flat(t, dtype, numel, name, on):
    """Pointer of a contiguous tensor of `numel` elements of `dtype` on the call's device (its index, not -1)."""
    if not (t.dtype is dtype and t.numel() == numel and t.get_device() == on and t.is_contiguous()):
        raise ValueError(f"{name}: a contiguous tensor of {numel} {dtype} values on the call's CUDA device is needed, "
                         f"got {tuple(t.shape)} {t.dtype} on {t.device}")
    return t.data_ptr()


def _matrix(t, dtype, rows, cols, name, on):
    """_flat for [rows, cols] (or its flat form): another shape of as many elements would be read in the wrong order."""
    at = _flat(t, dtype, rows * cols, name, on)
    if t.shape != (rows, cols) and t.dim() != 1 and rows > 1 and cols > 1:
        raise ValueError(f"{name}: the shape {[rows, cols]} is needed, got {list(t.shape)}")
    return at


def _dense_rows(t):
    """Whether the last dimension is contiguous (strides of empty and one-element dimensions mean nothing)."""
    return t.stride(-1) == 1 or t.shape[-1] <= 1 or t.numel() == 0


def _written(*tensors):
    """Tells autograd that a call has changed these (None: none). What it recorded on their values as they were raises in
    its backward pass, as after PyTorch's own changes in place."""
    for t in tensors:
        if t is not None:
            torch.autograd.graph.increment_version(t)


def _workspace_ptr(nbytes, device, workspace, stream, on):
    """Pointer and size of a call's workspace, and the tensor that holds it: the caller keeps that until the entry
    point has returned, or the allocator may hand the memory out before the last launch is queued."""
    if workspace is not None:
        size = workspace.numel() * workspace.element_size()
        _need(workspace.get_device() == on and workspace.is_contiguous(),
              "workspace: a contiguous tensor on the call's CUDA device is needed")
        _need(size >= nbytes, "workspace too small")
        return workspace.data_ptr(), size, workspace
    ws = _empty(nbytes, torch.uint8, device, stream)
    return ws.data_ptr(), nbytes, ws


# ---------------------------------------------------------------------------
# ak_batch_layout
# ---------------------------------------------------------------------------

def ak_batch_layout_workspace_size(nreq: int, opts=None) -> int:
    b = ctypes.c_size_t()
    _check(_abi.load().ak_batch_layout_workspace_size(int(nreq), _opts(opts), ctypes.byref(b)),
           "ak_batch_layout_workspace_size")
    return b.value


def ak_batch_layout(ctx_lens: torch.Tensor, new_lens: torch.Tensor, block_table: torch.Tensor,
                    free_blocks: torch.Tensor, *, block_size: int, max_tokens: int, offsets=None, slots=None,
                    positions=None, requests=None, counts=None, workspace=None, opts=None,
                    stream=None) -> BatchLayout:
    """Packed offsets, slot map, positions and request ids of a batch from its
    requests' int32 lengths (``ctx_lens`` cached, ``new_lens`` to run), and the
    new entries of ``block_table`` ([requests, width] int32, in place) taken in
    order from ``free_blocks``. Token arrays hold ``max_tokens`` entries, -1 / 0
    / -1 past the batch's end."""
    n, width = block_table.shape
    dev, on = ctx_lens.device, ctx_lens.get_device()
    if not (block_table.dtype is torch.int32 and block_table.get_device() == on >= 0 and _dense_rows(block_table)):
        raise ValueError("block_table: a [requests, width] int32 tensor with contiguous rows on the call's CUDA device is "
                         "needed")
    nfree = free_blocks.numel()
    inputs = (_flat(ctx_lens, torch.int32, n, "ctx_lens", on), _flat(new_lens, torch.int32, n, "new_lens", on),
              _flat(free_blocks, torch.int32, nfree, "free_blocks", on))
    p_off = p_slots = p_pos = p_req = p_cnt = None
    if offsets is None:
        offsets = _empty(n + 1, torch.int32, dev, stream)
    else:
        p_off = _flat(offsets, torch.int32, n + 1, "offsets", on)
    if slots is None:
        slots = _empty(max_tokens, torch.int64, dev, stream)
    else:
        p_slots = _flat(slots, torch.int64, max_tokens, "slots", on)
    if positions is None:
        positions = _empty(max_tokens, torch.int32, dev, stream)
    else:
        p_pos = _flat(positions, torch.int32, max_tokens, "positions", on)
    if requests is None:
        requests = _empty(max_tokens, torch.int32, dev, stream)
    else:
        p_req = _flat(requests, torch.int32, max_tokens, "requests", on)
    if counts is None:
        counts = _empty(2, torch.int32, dev, stream)
    else:
        p_cnt = _flat(counts, torch.int32, 2, "counts", on)
    # a single row's stride says nothing; rows that overlap are the entry point's to refuse
    stride = block_table.stride(0) if n > 1 else width
    wp, wb, _keep = None, 0, None
    if n > 4096 or workspace is not None:  # smaller batches need none
        wp, wb, _keep = _workspace_ptr(ak_batch_layout_workspace_size(n), dev, workspace, stream, on)
    _check(_abi.load().ak_batch_layout(
        inputs[0], inputs[1], n, block_table.data_ptr(), stride, width, inputs[2], nfree,
        block_size, max_tokens, p_off or offsets.data_ptr(), p_slots or slots.data_ptr(), p_pos or positions.data_ptr(),
        p_req or requests.data_ptr(), p_cnt or counts.data_ptr(), wp, wb, _opts(opts), _stream_of(stream, ctx_lens)),
        "ak_batch_layout")
    return BatchLayout(offsets, slots, positions, requests, counts)


# ---------------------------------------------------------------------------
# ak_verify_drafts
# ---------------------------------------------------------------------------

def ak_verify_drafts(target_probs: torch.Tensor, draft_tokens: torch.Tensor, uniform: torch.Tensor,
                     noise: torch.Tensor, *, draft_probs: torch.Tensor | None = None,
                     draft_counts: torch.Tensor | None = None, tokens: torch.Tensor | None = None,
                     accepted: torch.Tensor | None = None, opts=None, stream=None):
    """Verify ``draft_tokens`` [requests, k] int32 against ``target_probs``
    [requests, k + 1, vocab] (float32 or bfloat16) with ``uniform`` [requests, k]
    and exponential ``noise`` [requests, vocab]; ``draft_probs`` [requests, k,
    vocab] or None where each draft was certain. Returns ``(tokens, accepted)``:
    [requests, k + 1] int32, the kept drafts, then the token after them, then -1;
    and how many drafts were kept."""
    n, k = draft_tokens.shape
    vocab = target_probs.shape[-1]
    dev, dt, on = target_probs.device, target_probs.dtype, target_probs.get_device()
    kind = _FLOAT.get(dt)
    if kind is None:
        raise ValueError("probabilities are float32 or bfloat16")
    if not (target_probs.shape == (n, k + 1, vocab) and on >= 0 and _dense_rows(target_probs)):
        raise ValueError("target_probs: a [requests, k + 1, vocab] CUDA tensor with contiguous rows is needed")
    if not (noise.dtype is torch.float32 and noise.shape == (n, vocab) and noise.get_device() == on and _dense_rows(noise)):
        raise ValueError("noise: a [requests, vocab] float32 tensor with contiguous rows on the target's device is needed")
    q, qs = None, (0, 0)
    if draft_probs is not None:
        if not (draft_probs.dtype is dt and draft_probs.shape == (n, k, vocab) and draft_probs.get_device() == on and
                _dense_rows(draft_probs)):
            raise ValueError("draft_probs: a [requests, k, vocab] tensor of the target's type and device with "
                             "contiguous rows is needed")
        q, qs = (draft_probs.data_ptr() if k else None), draft_probs.stride()
    drafts = _flat(draft_tokens, torch.int32, n * k, "draft_tokens", on)
    u = _matrix(uniform, torch.float32, n, k, "uniform", on)
    m = None if draft_counts is None else _flat(draft_counts, torch.int32, n, "draft_counts", on)
    p_tok = p_acc = None
    if tokens is None:
        tokens = _empty((n, k + 1), torch.int32, dev, stream)
    else:
        p_tok = _matrix(tokens, torch.int32, n, k + 1, "tokens", on)
    if accepted is None:
        accepted = _empty(n, torch.int32, dev, stream)
    else:
        p_acc = _flat(accepted, torch.int32, n, "accepted", on)
    ps = target_probs.stride()
    _check(_abi.load().ak_verify_drafts(
        target_probs.data_ptr(), ps[0], ps[1], q, qs[0], qs[1], kind, drafts, m, u, noise.data_ptr(), noise.stride(0),
        n, k, vocab, p_tok or tokens.data_ptr(), p_acc or accepted.data_ptr(), _opts(opts),
        _stream_of(stream, target_probs)), "ak_verify_drafts")
    return tokens, accepted


# ---------------------------------------------------------------------------
# linear attention with a decay for each head
# ---------------------------------------------------------------------------

def _heads(t: torch.Tensor, shape, dtype, name, on) -> ak_heads:
    s = t.stride()
    if not (t.dtype is dtype and t.shape == shape and t.get_device() == on and (s[2] == 1 or shape[2] == 1)):
        raise ValueError(f"{name}: a {list(shape)} {dtype} tensor on q's CUDA device with a contiguous last dimension is "
                         f"needed, got {list(t.shape)} {t.dtype} with strides {list(s)} on {t.device}")
    return ak_heads(t.data_ptr(), s[0], s[1])


def _state_ptr(t, shape, name, on):
    if t is None:
        return None
    if not (t.get_device() == on and t.dtype == torch.float32 and t.shape == shape and t.is_contiguous()):
        raise ValueError(f"{name}: a contiguous {list(shape)} float32 tensor on q's CUDA device is needed, "
                         f"got {list(t.shape)} {t.dtype} on {t.device}")
    return t.data_ptr()


def _geometry(q, k, v, log_decay, offsets, scale, max_len):
    if q.dim() != 3 or v.dim() != 3:
        raise ValueError("q, k and v are [tokens, heads, dim] tensors")
    sk = q.shape
    t, h, dk = sk
    dv = v.shape[2]
    dt, on = q.dtype, q.get_device()
    kind = _FLOAT.get(dt)
    if kind is None or on < 0:
        raise ValueError("q, k and v are float32 or bfloat16 CUDA tensors")
    n, off = 1, None
    if offsets is not None:
        n = offsets.numel() - 1
        _need(n >= 0, "offsets: at least one value is needed")
        off = _flat(offsets, torch.int32, n + 1, "offsets", on)
    a = ak_linattn(t, n, max_len or 0, h, dk, dv, kind, scale, 0)
    ld = _flat(log_decay, torch.float32, h, "log_decay", on)
    return a, (t, h, dk), (t, h, dv), (n, h, dk, dv), dt, ld, off, on


def ak_linear_attention_workspace_size(tokens: int, heads: int, dk: int, dv: int, *, seqs: int = 1, max_len=None,
                                       dtype: str = "bf16", opts=None) -> int:
    b = ctypes.c_size_t()
    a = ak_linattn(tokens, seqs, int(max_len or 0), heads, dk, dv, DTYPES[dtype], 1.0, 0)
    _check(_abi.load().ak_linear_attention_workspace_size(ctypes.byref(a), _opts(opts), ctypes.byref(b)),
           "ak_linear_attention_workspace_size")
    return b.value


def _workspace(a, device, workspace, opts, stream, on):
    b = ctypes.c_size_t()
    _check(_abi.load().ak_linear_attention_workspace_size(a, opts, b), "ak_linear_attention_workspace_size")
    if b.value <= 256 and workspace is None and opts is None:
        return None, 0, None
    return _workspace_ptr(b.value, device, workspace, stream, on)


def _tracked(q, k, v, log_decay, state) -> bool:
    """Whether autograd records what is done with any of these."""
    return (q.requires_grad or k.requires_grad or v.requires_grad or log_decay.requires_grad or
            (state is not None and state.requires_grad)) and torch.is_grad_enabled()


class _Attention(torch.autograd.Function):
    """ak_linear_attention with its gradients in the graph."""

    @staticmethod
    def forward(ctx, q, k, v, log_decay, state, offsets, rest, final_state, workspace):
        ctx.save_for_backward(q, k, v, log_decay, state, offsets)
        ctx.rest = rest
        ctx.set_materialize_grads(False)
        return ak_linear_attention(q, k, v, log_decay, state=state, offsets=offsets, final_state=final_state,
                                   workspace=workspace, **rest)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, do, dstate_out):
        q, k, v, log_decay, state, offsets = ctx.saved_tensors
        if ctx.needs_input_grad[3]:
            raise RuntimeError("ak_linear_attention has no gradient for log_decay: pass log_decay.detach()")
        if do is None:
            do = torch.zeros_like(v)
        elif not _dense_rows(do):
            do = do.contiguous()
        dstate_out = None if dstate_out is None else dstate_out.contiguous()
        grads = ak_linear_attention_backward(do, q, k, v, log_decay, state=state, offsets=offsets, dstate_out=dstate_out,
                                             **ctx.rest)
        return (*grads[:3], None, grads[3], None, None, None, None)


class _Untracked(torch.autograd.Function):
    """Results of a call that has no gradient, for inputs that ask for one: a backward pass through them is an error."""

    @staticmethod
    def forward(ctx, results, why, *inputs):
        ctx.why = why
        return tuple(None if t is None else t.detach() for t in results)

    @staticmethod
    def backward(ctx, *_):
        raise RuntimeError(ctx.why)


def ak_linear_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, log_decay: torch.Tensor, *,
                        offsets: torch.Tensor | None = None, state: torch.Tensor | None = None, scale: float = 1.0,
                        max_len: int | None = None, out: torch.Tensor | None = None,
                        state_out: torch.Tensor | None = None, final_state: bool = False, workspace=None, opts=None,
                        stream=None):
    """``S_t = exp(log_decay) S_{t-1} + k_t v_t^T``, ``o_t = scale S_t^T q_t`` for
    every head over packed sequences (``offsets`` int32, None: one sequence),
    from ``state`` [sequences, heads, dk, dv] float32 or zero. Returns ``(out,
    state_out)``, the latter None unless given or asked for by ``final_state``.
    Gradients of q, k, v and ``state`` are recorded as usual, of results that the
    call allocates on the current stream; ``log_decay`` has none."""
    if _tracked(q, k, v, log_decay, state):
        if out is None and state_out is None and stream is None:
            return _Attention.apply(q, k, v, log_decay, state, offsets, dict(scale=scale, max_len=max_len, opts=opts),
                                    final_state, workspace)
        with torch.no_grad():
            results = ak_linear_attention(q, k, v, log_decay, offsets=offsets, state=state, scale=scale, max_len=max_len,
                                          out=out, state_out=state_out, final_state=final_state, workspace=workspace,
                                          opts=opts, stream=stream)
        return _Untracked.apply(results, "ak_linear_attention into given memory or on a given stream is not recorded: "
                                "no gradient", q, k, v, log_decay, state)
    a, sk, sv, ss, dt, ld, off, on = _geometry(q, k, v, log_decay, offsets, scale, max_len)
    if out is None:
        out = _empty(sv, dt, q.device, stream)
    if state_out is None and final_state:
        state_out = _empty(ss, torch.float32, q.device, stream)
    op = _opts(opts)
    hq, hk = _heads(q, sk, dt, "q", on), _heads(k, sk, dt, "k", on)
    hv, ho = _heads(v, sv, dt, "v", on), _heads(out, sv, dt, "out", on)
    s0, s1 = _state_ptr(state, ss, "state", on), _state_ptr(state_out, ss, "state_out", on)
    wp, wb, _keep = _workspace(a, q.device, workspace, op, stream, on)
    _check(_abi.load().ak_linear_attention(a, hq, hk, hv, ld, off, s0, ho, s1, wp, wb, op, _stream_of(stream, q)),
           "ak_linear_attention")
    return out, state_out


def ak_linear_attention_backward(do: torch.Tensor, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                                 log_decay: torch.Tensor, *, offsets: torch.Tensor | None = None,
                                 state: torch.Tensor | None = None, dstate_out: torch.Tensor | None = None,
                                 scale: float = 1.0, max_len: int | None = None, dq: torch.Tensor | None = None,
                                 dk: torch.Tensor | None = None, dv: torch.Tensor | None = None,
                                 dstate: torch.Tensor | None = None, workspace=None, opts=None, stream=None):
    """Gradients of ak_linear_attention with respect to q, k, v and the initial
    state, from the output's gradient ``do`` and the final state's
    ``dstate_out`` (or None). Returns ``(dq, dk, dv, dstate)``; ``dstate`` is
    None where the forward call had no ``state`` and none is given."""
    a, sk, sv, ss, dt, ld, off, on = _geometry(q, k, v, log_decay, offsets, scale, max_len)
    dev = q.device
    if dq is None:
        dq = _empty(sk, dt, dev, stream)
    if dk is None:
        dk = _empty(sk, dt, dev, stream)
    if dv is None:
        dv = _empty(sv, dt, dev, stream)
    if dstate is None and state is not None:
        dstate = _empty(ss, torch.float32, dev, stream)
    op = _opts(opts)
    hs = [_heads(x, s, dt, n, on) for x, s, n in ((do, sv, "do"), (q, sk, "q"), (k, sk, "k"), (v, sv, "v"),
                                              (dq, sk, "dq"), (dk, sk, "dk"), (dv, sv, "dv"))]
    hdo, hq, hk, hv, hdq, hdk, hdv = hs
    s0, s1 = _state_ptr(state, ss, "state", on), _state_ptr(dstate_out, ss, "dstate_out", on)
    s2 = _state_ptr(dstate, ss, "dstate", on)
    wp, wb, _keep = _workspace(a, dev, workspace, op, stream, on)
    _check(_abi.load().ak_linear_attention_backward(a, hdo, hq, hk, hv, ld, off, s0, s1, hdq, hdk, hdv,
                                                    s2, wp, wb, op, _stream_of(stream, q)),
           "ak_linear_attention_backward")
    return dq, dk, dv, dstate


def ak_linear_attention_step(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, log_decay: torch.Tensor,
                             state: torch.Tensor, *, slots: torch.Tensor | None = None, scale: float = 1.0,
                             out: torch.Tensor | None = None, opts=None, stream=None) -> torch.Tensor:
    """One token of each of ``q.shape[0]`` requests: updates the matrices
    ``state[slots]`` ([slots, heads, dk, dv] float32; ``slots`` int32, None: request
    b uses state[b]) in place and returns the outputs. Slots outside the pool
    mark padding and give zeros. It has no gradient."""
    if _tracked(q, k, v, log_decay, state):
        with torch.no_grad():
            out = ak_linear_attention_step(q, k, v, log_decay, state, slots=slots, scale=scale, out=out, opts=opts,
                                           stream=stream)
        return _Untracked.apply((out,), "ak_linear_attention_step has no gradient", q, k, v, log_decay, state)[0]
    a, sk, sv, ss, dt, ld, _, on = _geometry(q, k, v, log_decay, None, scale, None)
    if out is None:
        out = _empty(sv, dt, q.device, stream)
    hq, hk = _heads(q, sk, dt, "q", on), _heads(k, sk, dt, "k", on)
    hv, ho = _heads(v, sv, dt, "v", on), _heads(out, sv, dt, "out", on)
    pool = state.shape[0]
    sp = _state_ptr(state, (pool,) + ss[1:], "state", on)
    at = None if slots is None else _flat(slots, torch.int32, sk[0], "slots", on)
    _need(slots is not None or pool >= sk[0], "state: one matrix for each request and head is needed")
    _check(_abi.load().ak_linear_attention_step(a, hq, hk, hv, ld, sp, at, pool, ho, _opts(opts),
                                                _stream_of(stream, q)),
           "ak_linear_attention_step")
    return out
