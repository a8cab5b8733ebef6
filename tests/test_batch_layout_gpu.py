"""ak_batch_layout against the request-by-request definition: whole numbers, so exactly."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import mapreduce_prefix_scan_gb300 as ak
from sequence_reference import layout

pytestmark = pytest.mark.gpu


def _case(rng, n, top_ctx, top_new, block, width=None):
    ctx = rng.integers(0, top_ctx + 1, n)
    new = rng.integers(0, top_new + 1, n)
    have = -(-ctx // block)
    width = width or int((-(-(ctx + new) // block)).max(initial=1)) + 1
    ids = rng.permutation(int(have.sum()) + int((-(-(ctx + new) // block) - have).sum()) + 3)
    table = np.full((n, width), -1, np.int64)
    at = 0
    for r in range(n):
        m = min(int(have[r]), width)
        table[r, :m] = ids[at:at + m]
        at += int(have[r])
    return ctx, new, table, ids[at:]


def _run(ctx, new, table, free, block, max_tokens, table_view=None, **kw):
    t = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")
    dev = t(table) if table_view is None else table_view
    r = ak.ak_batch_layout(t(ctx), t(new), dev, t(free), block_size=block, max_tokens=max_tokens, **kw)
    return [x.cpu().numpy() for x in (r.offsets, r.slots, r.positions, r.requests, r.counts, dev)]


def _same(got, want):
    for name, a, b in zip(("offsets", "slots", "positions", "requests", "counts", "table"), got, want):
        assert np.array_equal(a, b), name


@pytest.mark.parametrize("n,top_ctx,top_new,block", [
    (1, 0, 1, 16), (1, 40, 5000, 16), (7, 100, 0, 16), (33, 90, 3, 1), (64, 1000, 200, 24),
    (300, 50, 1, 16), (2047, 70, 9, 7), (4096, 20, 3, 16), (4097, 20, 3, 16), (9000, 9, 5, 32)])
@pytest.mark.parametrize("room", [0, 1, 6])
def test_against_definition(n, top_ctx, top_new, block, room):
    rng = np.random.default_rng(n + block)
    ctx, new, table, free = _case(rng, n, top_ctx, top_new, block)
    most = int(new.sum()) + room
    _same(_run(ctx, new, table, free, block, most), layout(ctx, new, table, free, block, most))


def test_long_runs_of_empty_requests():
    rng = np.random.default_rng(5)
    ctx, new, table, free = _case(rng, 700, 60, 9, 16)
    new[:250] = 0
    new[300:699] = 0
    _same(_run(ctx, new, table, free, 16, 120), layout(ctx, new, table, free, 16, 120))


def test_what_does_not_fit_is_left_out():
    rng = np.random.default_rng(6)
    ctx, new, table, free = _case(rng, 40, 100, 60, 16, width=6)   # some requests outgrow the table
    total = int(new.sum())
    for most, blocks in ((total // 2, len(free)), (total, len(free) // 3), (total, 0)):
        _same(_run(ctx, new, table, free[:blocks], 16, most), layout(ctx, new, table, free[:blocks], 16, most))


def test_negative_lengths_and_unset_blocks():
    ctx, new = np.array([20, -5, 8, 31]), np.array([3, 4, -2, 2])
    table = np.array([[4, -1, 9], [-1, -1, -1], [2, -1, -1], [-1, 7, -1]])  # block 1 of request 0 was never set
    _same(_run(ctx, new, table, [11, 12, 13], 16, 12), layout(ctx, new, table, [11, 12, 13], 16, 12))


def test_strided_table_and_unaligned_outputs():
    rng = np.random.default_rng(7)
    ctx, new, table, free = _case(rng, 50, 100, 30, 16)
    wide = torch.full((50, table.shape[1] + 5), -7, dtype=torch.int32, device="cuda")
    view = wide[:, 2:2 + table.shape[1]]
    view.copy_(torch.tensor(table, dtype=torch.int32))
    most = int(new.sum()) + 3
    off = lambda dt: torch.empty(most + 1, dtype=dt, device="cuda")[1:]
    got = _run(ctx, new, table, free, 16, most, table_view=view, slots=off(torch.int64),
               positions=off(torch.int32), requests=off(torch.int32))
    _same(got, layout(ctx, new, table, free, 16, most))
    assert (wide[:, :2] == -7).all() and (wide[:, -3:] == -7).all()


def test_no_requests_and_no_tokens():
    z = torch.empty(0, dtype=torch.int32, device="cuda")
    r = ak.ak_batch_layout(z, z, torch.empty(0, 4, dtype=torch.int32, device="cuda"), z, block_size=16, max_tokens=5)
    assert r.offsets.tolist() == [0] and r.counts.tolist() == [0, 0]
    assert r.slots.tolist() == [-1] * 5 and r.requests.tolist() == [-1] * 5 and r.positions.tolist() == [0] * 5
    one = torch.ones(3, dtype=torch.int32, device="cuda")
    r = ak.ak_batch_layout(one, one, torch.zeros(3, 2, dtype=torch.int32, device="cuda"), z, block_size=16, max_tokens=0)
    assert r.offsets.tolist() == [0, 1, 2, 3] and r.counts.tolist() == [3, 0]


def test_another_stream_and_a_graph_on_new_lengths():
    rng = np.random.default_rng(8)
    ctx, new, table, free = _case(rng, 90, 100, 12, 16)
    t = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")
    c, m, tb, f = t(ctx), t(new), t(table), t(free)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    r = ak.ak_batch_layout(c, m, tb.clone(), f, block_size=16, max_tokens=1200, stream=side)
    side.synchronize()
    assert np.array_equal(r.slots.cpu().numpy(), layout(ctx, new, table, free, 16, 1200)[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        r = ak.ak_batch_layout(c, m, tb, f, block_size=16, max_tokens=1200)
    new2 = rng.permutation(new)
    table2 = np.where(np.arange(table.shape[1])[None] < (-(-ctx // 16))[:, None], table, -1)
    m.copy_(t(new2))
    tb.copy_(t(table2))
    g.replay()
    torch.cuda.synchronize()
    width = max(table.shape[1], 1)
    want = layout(ctx, new2, table2[:, :width], free, 16, 1200)
    assert np.array_equal(r.slots.cpu().numpy(), want[1]) and np.array_equal(tb.cpu().numpy(), want[5])
