"""Beam search and the blocks of a paged cache over torch tensors.

These functions only marshal arguments; include/ak.h states the rules of
every argument.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple

import torch

from . import _abi
from . import sequence as _s


class BeamStep(NamedTuple):
    """A request's beams after a step, ``[requests, beams]`` each: ``parents`` is the beam that each one extends."""
    scores: torch.Tensor
    tokens: torch.Tensor
    parents: torch.Tensor
    done: torch.Tensor
    lengths: torch.Tensor


class BlockFork(NamedTuple):
    """What ak_blocks_fork makes: ``pairs`` are the blocks to copy (from, to), ``counts`` holds how many were wanted."""
    table: torch.Tensor
    lens: torch.Tensor
    refs: torch.Tensor
    pairs: torch.Tensor
    counts: torch.Tensor


def _given(t, shape, dtype, name, on, device, stream):
    """An output: the tensor given for it, or a new one."""
    if t is None:
        return _s._empty(shape, dtype, device, stream)
    if not (t.dtype is dtype and t.shape == shape and t.get_device() == on and t.is_contiguous()):
        raise ValueError(f"{name}: a contiguous {list(shape)} {dtype} tensor on the call's CUDA device is needed, "
                         f"got {list(t.shape)} {t.dtype} on {t.device}")
    return t


def _shaped(t, shape, dtype, name, on):
    """Pointer of a contiguous input of this shape; None for None."""
    return None if t is None else _given(t, shape, dtype, name, on, None, None).data_ptr()


def _int32(v, name):
    """A number that the entry point takes as an int32: ctypes would hand over its low bits."""
    if not -(1 << 31) <= v < 1 << 31:
        raise ValueError(f"{name}: {v} is out of range")
    return v


# ---------------------------------------------------------------------------
# beam search
# ---------------------------------------------------------------------------

def ak_beam_select(logits: torch.Tensor, scores: torch.Tensor, *, done: torch.Tensor | None = None,
                   lengths: torch.Tensor | None = None, end_token: int = -1, length_penalty: float = 0.0,
                   keep: int | None = None, out: BeamStep | None = None, opts=None, stream=None) -> BeamStep:
    """One step of a beam search: of every request's ``logits`` [requests, beams,
    vocab] (float32 or bfloat16) and its beams' summed log probabilities ``scores``
    [requests, beams] the best ``keep`` (default: as many as there are beams)
    continuations by total over length**``length_penalty``, ties by the lowest beam, then
    token. Beams that are ``done`` (bool) go on as they are, by ``end_token``. ``lengths``
    (int32) are the beams' tokens so far. ``out`` reuses an earlier step's tensors, which may be this
    step's inputs. It has no gradient."""
    if (logits.requires_grad or scores.requires_grad) and torch.is_grad_enabled():
        with torch.no_grad():
            step = ak_beam_select(logits, scores, done=done, lengths=lengths, end_token=end_token, length_penalty=length_penalty,
                                  keep=keep, out=out, opts=opts, stream=stream)
        return BeamStep(*_s._Untracked.apply(step, "ak_beam_select has no gradient", logits, scores))
    if logits.dim() != 3:
        raise ValueError("logits are [requests, beams, vocab]")
    n, k, vocab = logits.shape
    dt, dev, on = logits.dtype, logits.device, logits.get_device()
    kind = _s._FLOAT.get(dt)
    if kind is None or on < 0 or not _s._dense_rows(logits):
        raise ValueError("logits: a float32 or bfloat16 CUDA tensor with contiguous rows is needed")
    m = k if keep is None else _int32(int(keep), "keep")
    _int32(end_token, "end_token")
    if out is None:  # (allocations are half of a small call's time, views of a larger one more)
        e, shape, i32 = _s._empty, (n, m), torch.int32
        step = BeamStep(e(shape, torch.float32, dev, stream), e(shape, i32, dev, stream), e(shape, i32, dev, stream),
                        e(shape, torch.bool, dev, stream), e(shape, i32, dev, stream))
    else:
        step = BeamStep(*(_given(t, (n, m), d, f, on, dev, stream) for t, d, f in zip(
            out, (torch.float32, torch.int32, torch.int32, torch.bool, torch.int32), BeamStep._fields)))
    ls = logits.stride()
    _s._check(_abi.load().ak_beam_select(
        logits.data_ptr(), ls[0], ls[1], kind, n, k, vocab, m, _shaped(scores, (n, k), torch.float32, "scores", on),
        _shaped(done, (n, k), torch.bool, "done", on), _shaped(lengths, (n, k), torch.int32, "lengths", on), end_token,
        length_penalty, *(t.data_ptr() for t in step), _s._opts(opts), _s._stream_of(stream, logits)), "ak_beam_select")
    if out is not None:
        _s._written(*step)
    return step


def _leading(t, dim, name):
    """The dimensions before `dim` as one: (count, stride in bytes)."""
    if dim < 0 or dim >= t.dim():
        raise ValueError(f"{name}: dim is out of range")
    count, stride, e = 1, 0, t.element_size()
    for i in reversed(range(dim)):
        if t.shape[i] == 1:
            continue
        if count > 1 and t.stride(i) != stride * count:
            raise ValueError(f"{name}: the dimensions before dim {dim} do not lie at one stride")
        if count == 1:
            stride = t.stride(i)
        count *= t.shape[i]
    return count, stride * e


def _inner(t, dim, name):
    """Bytes of the dimensions from `dim` on, which are contiguous."""
    size = 1
    for i in reversed(range(dim, t.dim())):
        if t.shape[i] != 1 and t.stride(i) != size:
            raise ValueError(f"{name}: the dimensions from {dim} on are not contiguous")
        size *= t.shape[i]
    return size * t.element_size()


def _no_grad_in_place(t, name):
    if t.requires_grad and torch.is_grad_enabled():
        raise RuntimeError(f"{name} changes its tensor in place and has no gradient: pass it detached")


def ak_beam_reorder(state: torch.Tensor, parents: torch.Tensor, *, dim: int = 0, opts=None, stream=None) -> torch.Tensor:
    """``state[..., r, k, ...] = state[..., r, parents[r, k], ...]`` in place, with
    requests along ``dim`` and beams along ``dim + 1`` of a tensor of any type.
    ``parents`` [requests, beams] int32 as ak_beam_select gives them; a beam whose parent is
    outside the beams keeps its own. Returns ``state``."""
    _no_grad_in_place(state, "ak_beam_reorder")
    if dim < 0 or state.dim() < dim + 2:
        raise ValueError("state: requests along dim and beams along dim + 1 are needed")
    n, k = state.shape[dim], state.shape[dim + 1]
    on, e = state.get_device(), state.element_size()
    if on < 0:
        raise ValueError("state: a CUDA tensor is needed")
    if state.numel() == 0:
        return state
    outer, outer_stride = _leading(state, dim, "state")
    inner = _inner(state, dim + 2, "state") if state.dim() > dim + 2 else e
    p = _shaped(parents, (n, k), torch.int32, "parents", on)
    _s._check(_abi.load().ak_beam_reorder(state.data_ptr(), outer, outer_stride, n, state.stride(dim) * e, k,
                                          state.stride(dim + 1) * e, inner, p, _s._opts(opts),
                                          _s._stream_of(stream, state)), "ak_beam_reorder")
    _s._written(state)
    return state


# ---------------------------------------------------------------------------
# blocks of a paged cache
# ---------------------------------------------------------------------------

def _table(block_table, lens, block_size, on):
    """Arguments of a block table and its requests' lengths."""
    _int32(block_size, "block_size")
    if not (block_table.dim() == 2 and block_table.dtype is torch.int32 and block_table.get_device() == on >= 0 and
            _s._dense_rows(block_table)):
        raise ValueError("block_table: a [requests, width] int32 tensor with contiguous rows on the call's CUDA device is needed")
    n, width = block_table.shape
    return (block_table.data_ptr(), block_table.stride(0) if n > 1 else width, width, _s._flat(lens, torch.int32, n, "lens", on), n)


def ak_blocks_count(block_table: torch.Tensor, lens: torch.Tensor, *, block_size: int, blocks: int,
                    out: torch.Tensor | None = None, opts=None, stream=None) -> torch.Tensor:
    """How many requests hold each of the pool's ``blocks`` ([blocks] int32): the
    first ceil(len / block_size) entries of each request's row of ``block_table``."""
    on = block_table.get_device()
    a = _table(block_table, lens, block_size, on)
    if out is None:
        refs = _s._empty(blocks, torch.int32, block_table.device, stream)
    else:
        refs = _given(out, (blocks,), torch.int32, "out", on, None, None)
    _s._check(_abi.load().ak_blocks_count(*a, block_size, blocks, refs.data_ptr(), _s._opts(opts),
                                          _s._stream_of(stream, block_table)), "ak_blocks_count")
    _s._written(out)
    return refs


def ak_blocks_fork_workspace_size(rows: int, blocks: int, opts=None) -> int:
    """Bytes of the ``workspace`` of a fork into ``rows`` requests over a pool of ``blocks``."""
    b = ctypes.c_size_t()
    _s._check(_abi.load().ak_blocks_fork_workspace_size(int(rows), int(blocks), _s._opts(opts), ctypes.byref(b)),
              "ak_blocks_fork_workspace_size")
    return b.value


def ak_blocks_compact_workspace_size(blocks: int, opts=None) -> int:
    """Bytes of the ``workspace`` of a compaction of a pool of ``blocks``."""
    b = ctypes.c_size_t()
    _s._check(_abi.load().ak_blocks_compact_workspace_size(int(blocks), _s._opts(opts), ctypes.byref(b)),
              "ak_blocks_compact_workspace_size")
    return b.value


def ak_blocks_fork(block_table: torch.Tensor, lens: torch.Tensor, parents: torch.Tensor, free_blocks: torch.Tensor, *,
                   block_size: int, blocks: int, out: BlockFork | None = None, workspace=None, opts=None,
                   stream=None) -> BlockFork:
    """Requests that go on from others: row r of the result from row
    ``parents[r]`` of ``block_table`` (an empty row for a parent outside it).
    Requests that end in the same partly filled block get their own, in order from ``free_blocks``;
    ``pairs`` lists what ak_blocks_copy has to copy. ``refs`` are the counts of the result.
    ``out`` reuses an earlier fork's tensors, not those of the input."""
    on, dev = block_table.get_device(), block_table.device
    a = _table(block_table, lens, block_size, on)
    n, nfree = parents.numel(), free_blocks.numel()
    p, fb = _s._flat(parents, torch.int32, n, "parents", on), _s._flat(free_blocks, torch.int32, nfree, "free_blocks", on)
    width = block_table.shape[1]
    if out is None:
        e, i32 = _s._empty, torch.int32
        f = BlockFork(e((n, width), i32, dev, stream), e(n, i32, dev, stream), e(blocks, i32, dev, stream), e((n, 2), i32, dev, stream),
                      e(1, i32, dev, stream))
    else:
        f = BlockFork(*(_given(t, s, torch.int32, name, on, dev, stream) for t, s, name in zip(
            out, ((n, width), (n,), (blocks,), (n, 2), (1,)), BlockFork._fields)))
    b = ctypes.c_size_t()
    L = _abi.load()
    _s._check(L.ak_blocks_fork_workspace_size(n, blocks, None, b), "ak_blocks_fork_workspace_size")
    wp, wb, _keep = _s._workspace_ptr(b.value, dev, workspace, stream, on)
    _s._check(L.ak_blocks_fork(*a, p, n, fb, nfree, block_size, blocks, f.table.data_ptr(), width, f.lens.data_ptr(),
                               f.refs.data_ptr(), f.pairs.data_ptr(), f.counts.data_ptr(), wp, wb, _s._opts(opts),
                               _s._stream_of(stream, block_table)), "ak_blocks_fork")
    if out is not None:
        _s._written(*f)
    return f


def ak_blocks_free(refs: torch.Tensor, *, out: torch.Tensor | None = None, counts: torch.Tensor | None = None, opts=None,
                   stream=None):
    """The blocks that nobody holds: ``(free_blocks, counts)``, their ids in increasing
    order, then -1 ([blocks] int32), and how many they are ([1] int32)."""
    on, n = refs.get_device(), refs.numel()
    p = _s._flat(refs, torch.int32, n, "refs", on)
    dev, given = refs.device, (out, counts)
    free = _s._empty(n, torch.int32, dev, stream) if out is None else _given(out, (n,), torch.int32, "out", on, dev, stream)
    counts = _s._empty(1, torch.int32, dev, stream) if counts is None else _given(counts, (1,), torch.int32, "counts", on, dev, stream)
    _s._check(_abi.load().ak_blocks_free(p, n, free.data_ptr(), counts.data_ptr(), _s._opts(opts), _s._stream_of(stream, refs)),
              "ak_blocks_free")
    _s._written(*given)
    return free, counts


def ak_blocks_compact(block_table: torch.Tensor, lens: torch.Tensor, refs: torch.Tensor, *, block_size: int,
                      out: torch.Tensor | None = None, pairs: torch.Tensor | None = None,
                      counts: torch.Tensor | None = None, workspace=None, opts=None, stream=None):
    """Packs the blocks in use (``refs`` of ak_blocks_count) to the pool's front:
    ``(table, pairs, counts)``, the table with its blocks renamed (``out`` may be
    ``block_table``), the (from, to) that ak_blocks_copy has to copy, then (-1, -1), and [moves, blocks in
    use]."""
    on, dev, given = block_table.get_device(), block_table.device, (out, pairs, counts)
    a = _table(block_table, lens, block_size, on)
    blocks = refs.numel()
    rp = _s._flat(refs, torch.int32, blocks, "refs", on)
    if out is block_table:
        table, stride = out, a[1]
    else:
        table, stride = _given(out, block_table.shape, torch.int32, "out", on, dev, stream), a[2]
    pairs = _given(pairs, (blocks // 2, 2), torch.int32, "pairs", on, dev, stream)
    counts = _given(counts, (2,), torch.int32, "counts", on, dev, stream)
    b = ctypes.c_size_t()
    L = _abi.load()
    _s._check(L.ak_blocks_compact_workspace_size(blocks, None, b), "ak_blocks_compact_workspace_size")
    wp, wb, _keep = _s._workspace_ptr(b.value, dev, workspace, stream, on)
    _s._check(L.ak_blocks_compact(*a, rp, block_size, blocks, table.data_ptr(), stride, pairs.data_ptr(), counts.data_ptr(),
                                  wp, wb, _s._opts(opts), _s._stream_of(stream, block_table)), "ak_blocks_compact")
    _s._written(*given)
    return table, pairs, counts


def ak_blocks_copy(cache: torch.Tensor, pairs: torch.Tensor, *, counts: torch.Tensor | None = None, dim: int = 0, opts=None,
                   stream=None) -> torch.Tensor:
    """Copies blocks of ``cache`` (of any type, blocks along ``dim``) in place: for each of
    ``pairs`` [n, 2] int32, ``cache[..., to] = cache[..., from]``. ``counts[0]`` (device) bounds how many are
    looked at. Returns ``cache``."""
    _no_grad_in_place(cache, "ak_blocks_copy")
    on = cache.get_device()
    if on < 0:
        raise ValueError("cache: a CUDA tensor is needed")
    outer, outer_stride = _leading(cache, dim, "cache")
    n = pairs.shape[0]
    p = _shaped(pairs, (n, 2), torch.int32, "pairs", on)
    c = None if counts is None else _s._flat(counts, torch.int32, counts.numel(), "counts", on)
    if counts is not None and counts.numel() < 1:
        raise ValueError("counts: at least one value is needed")
    if cache.numel() == 0:
        return cache
    e = cache.element_size()
    inner = _inner(cache, dim + 1, "cache") if cache.dim() > dim + 1 else e
    _s._check(_abi.load().ak_blocks_copy(cache.data_ptr(), outer, outer_stride, cache.shape[dim], cache.stride(dim) * e, inner, p,
                                         n, c, _s._opts(opts), _s._stream_of(stream, cache)), "ak_blocks_copy")
    _s._written(cache)
    return cache
