"""Block operators against their definitions: whole numbers, so equal."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import decoding_reference as ref
import mapreduce_prefix_scan_gb300 as ak

pytestmark = pytest.mark.gpu


def _i(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def _pool(n, width, block, blocks, seed, shared=0.5):
    """Requests with random lengths, some prefixes shared; returns table, lens and the ids left."""
    rng = np.random.default_rng(seed)
    ids = list(rng.permutation(blocks))
    table, lens = np.full((n, width), -1), np.zeros(n, int)
    for r in range(n):
        lens[r] = rng.integers(0, width * block + 1)
        nb = -(-lens[r] // block)
        same = 0
        if r and rng.random() < shared:
            same = min(nb, int(lens[r - 1] // block))  # full blocks of the one before
            table[r, :same] = table[r - 1, :same]
        if nb - same > len(ids):
            nb, lens[r] = same, same * block
        for c in range(same, nb):
            table[r, c] = ids.pop()
        table[r, nb:] = rng.integers(-5, blocks + 5, width - nb)  # what lies past a request's blocks means nothing
    return table, lens, np.array(ids, int)


SIZES = [(1, 1, 1, 4), (3, 5, 16, 40), (8, 38, 16, 400), (64, 40, 8, 3000), (200, 130, 24, 30000), (5, 1000, 1, 6000)]


@pytest.mark.parametrize("n,width,block,blocks", SIZES)
def test_count_and_free(n, width, block, blocks):
    table, lens, _ = _pool(n, width, block, blocks, n)
    refs = ak.ak_blocks_count(_i(table), _i(lens), block_size=block, blocks=blocks)
    want = ref.count(table, lens, block, blocks)
    assert refs.tolist() == want.tolist()
    free, counts = ak.ak_blocks_free(refs)
    ids, m = ref.free_list(want)
    assert free.tolist() == ids.tolist() and counts.tolist() == m.tolist()


@pytest.mark.parametrize("blocks", [1, 31, 1024, 1025, 16384, 100003, 1000000])
@pytest.mark.parametrize("share", [0.0, 0.4, 1.0])
def test_free_of_any_size(blocks, share):
    refs = (np.random.default_rng(blocks).random(blocks) < share).astype(int) * 3
    refs[::7] -= 2  # a count below zero is none
    free, counts = ak.ak_blocks_free(_i(refs))
    ids, m = ref.free_list(refs)
    assert counts.tolist() == m.tolist() and (free.cpu().numpy() == ids).all()


def _fork(table, lens, parents, free, block, blocks, **kw):
    f = ak.ak_blocks_fork(_i(table), _i(lens), _i(parents), _i(free), block_size=block, blocks=blocks, **kw)
    want = ref.fork(np.asarray(table), lens, parents, free, block, blocks)
    for name, got, w in zip(f._fields, f, want):
        assert got.tolist() == w.tolist(), name
    # the counts are those of the result
    assert f.refs.tolist() == ref.count(f.table.cpu().numpy(), f.lens.tolist(), block, blocks).tolist()
    return f


@pytest.mark.parametrize("seed", range(3))
@pytest.mark.parametrize("n,width,block,blocks", SIZES)
def test_fork(n, width, block, blocks, seed):
    table, lens, free = _pool(n, width, block, blocks, 10 * n + seed)
    rng = np.random.default_rng(seed)
    for new in (n, max(1, n // 2), 2 * n + 1):
        parents = rng.integers(-1, n + 1, new)
        _fork(table, lens, parents, free, block, blocks)
    _fork(table, lens, np.arange(n), free, block, blocks)
    _fork(table, lens, np.full(n, n - 1), free, block, blocks)


def test_fork_shares_a_partial_block_only_until_it_is_written():
    # block 4: row 0 holds 6 tokens (blocks 10, 11), row 1 eight (blocks 10, 12)
    table, lens = [[10, 11, -1], [10, 12, -1]], [6, 8]
    f = _fork(table, lens, [0, 0, 1, 1], [3, 7, 9], 4, 16)
    assert f.table.tolist() == [[10, 11, -1], [10, 3, -1], [10, 12, -1], [10, 12, -1]] and f.pairs.tolist()[0] == [11, 3]
    # a request that holds all of the block keeps it from both
    f = _fork([[10, 11], [10, 11]], [6, 8], [0, 0, 1], [3, 7, 9], 4, 16)
    assert f.pairs.tolist()[:2] == [[11, 3], [11, 7]] and f.table[2].tolist() == [10, 11]


def test_fork_past_the_free_list():
    table, lens = [[1, 2]], [5]
    f = _fork(table, lens, [0, 0, 0, 0], [7, -1], 4, 8)
    assert f.counts.tolist() == [3] and f.pairs.tolist() == [[2, 7], [-1, -1], [-1, -1], [-1, -1]]
    _fork(table, lens, [0, 0], [], 4, 8)
    _fork(table, lens, [0, 0, 0], [99, 3], 4, 8)
    # the padded list of ak_blocks_free
    free, _ = ak.ak_blocks_free(ak.ak_blocks_count(_i(table), _i(lens), block_size=4, blocks=8))
    _fork(table, lens, [0] * 9, free.tolist(), 4, 8)


def test_bad_entries_hold_nothing():
    table = [[5, -3, 100, 2], [2, 5, 2, 2], [7, 8, 1 << 30, 0]]
    lens = [15, 14, 1000]  # the last one past the table
    refs = ak.ak_blocks_count(_i(table), _i(lens), block_size=4, blocks=9)
    assert refs.tolist() == ref.count(np.array(table), lens, 4, 9).tolist()
    _fork(table, lens, [0, 0, 1, 2, 1, -7, 3], [3, 4, 6], 4, 9)
    assert ak.ak_blocks_count(_i(table), _i([-4, 0, -2147483648]), block_size=4, blocks=9).sum() == 0


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("n,width,block,blocks", SIZES)
def test_compact(n, width, block, blocks, in_place):
    table, lens, _ = _pool(n, width, block, blocks, n + 77)
    refs = ak.ak_blocks_count(_i(table), _i(lens), block_size=block, blocks=blocks)
    t = _i(table)
    out, pairs, counts = ak.ak_blocks_compact(t, _i(lens), refs, block_size=block, out=t if in_place else None)
    want = ref.compact(table, lens, refs.tolist(), block)
    assert (out is t) == in_place
    for got, w in zip((out, pairs, counts), want):
        assert got.tolist() == w.tolist()
    # again there is nothing to do
    refs = ak.ak_blocks_count(out, _i(lens), block_size=block, blocks=blocks)
    again, pairs, counts = ak.ak_blocks_compact(out, _i(lens), refs, block_size=block)
    assert torch.equal(again, out) and counts.tolist()[0] == 0 and (pairs == -1).all()


@pytest.mark.parametrize("blocks", [1, 2, 1023, 50000, 300001])
def test_compact_of_any_pattern(blocks):
    rng = np.random.default_rng(blocks)
    for share in (0.0, 0.1, 0.5, 0.95, 1.0):
        refs = (rng.random(blocks) < share).astype(int)
        table, lens = np.flatnonzero(refs)[:64][None], [64]
        out, pairs, counts = ak.ak_blocks_compact(_i(table), _i(lens), _i(refs), block_size=1)
        want = ref.compact(table, lens, refs.tolist(), 1)
        assert counts.tolist() == want[2].tolist() and (pairs.cpu().numpy() == want[1]).all() and out.tolist() == want[0].tolist()


@pytest.mark.parametrize("dtype,page", [(torch.bfloat16, (16, 2, 64)), (torch.float32, (3,)), (torch.uint8, (5, 7)), (torch.int64, ()),
                                        (torch.bfloat16, (70, 8, 64))])
@pytest.mark.parametrize("layers", [0, 1, 3])
def test_copy(dtype, page, layers):
    g = torch.Generator().manual_seed(1)
    shape = ((layers,) if layers else ()) + (50,) + page
    cache = torch.randint(0, 100, shape, generator=g).to(dtype).cuda()
    pairs = _i([[3, 40], [3, 41], [7, 42], [-1, -1], [49, 0], [50, 1], [2, -1], [5, 5], [9, 12]])
    dim = 1 if layers else 0
    for count in (None, 0, 2, 9, 100, -3):
        want = cache.clone()
        w = want if layers else want[None]
        for a, b in pairs.tolist()[: 9 if count is None else max(count, 0)]:
            if 0 <= a < 50 and 0 <= b < 50:
                w[:, b] = w[:, a]
        got = cache.clone()
        ak.ak_blocks_copy(got, pairs, counts=None if count is None else _i([count, 5]), dim=dim)
        assert torch.equal(got, want), count


def test_copy_in_views():
    """Keys and values of one tensor, a slice of the heads, blocks apart."""
    cache = torch.randn(2, 30, 2, 8, 16, device="cuda")  # [layer, block, k or v, ...]
    pairs = _i([[1, 20], [2, 21]])
    want = cache.clone()
    want[:, [20, 21], 1] = cache[:, [1, 2], 1]
    ak.ak_blocks_copy(cache[:, :, 1], pairs, dim=1)
    assert torch.equal(cache, want)
    with pytest.raises(ValueError):
        ak.ak_blocks_copy(cache.transpose(3, 4), pairs, dim=1)
    with pytest.raises(ValueError):
        ak.ak_blocks_copy(torch.zeros(3, 4, 30, 8, device="cuda")[:, :2], pairs, dim=2)


def test_copy_past_two_to_the_32_bytes():
    cache = torch.empty(5000, 1 << 20, dtype=torch.uint8, device="cuda")
    cache[4999], cache[3] = 7, 9
    ak.ak_blocks_copy(cache, _i([[4999, 4998], [3, 4997]]))
    assert (cache[4998] == 7).all() and (cache[4997] == 9).all()


def test_captured_decoding_step_replays():
    """Fork, copy and the free list in one graph, on new parents each time; two graphs with workspaces of their own."""
    n, width, block, blocks = 24, 12, 8, 600
    table, lens, free = _pool(n, width, block, blocks, 5, shared=0.0)
    t, m, fr, parents = _i(table), _i(lens), _i(free), _i(np.arange(n))
    cache = torch.randint(0, 1000, (blocks, block), device="cuda")

    def call():
        f = ak.ak_blocks_fork(t, m, parents, fr, block_size=block, blocks=blocks)
        ak.ak_blocks_copy(cache, f.pairs, counts=f.counts)
        return f, ak.ak_blocks_free(f.refs)

    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        f, (ids, count) = call()
    for seed in range(4):
        p = np.random.default_rng(seed).integers(-1, n, n)
        parents.copy_(_i(p))
        before = cache.clone()
        g.replay()
        want = ref.fork(table, lens, p, free, block, blocks)
        assert all(got.tolist() == w.tolist() for got, w in zip(f, want))
        assert ids.tolist() == ref.free_list(want[2])[0].tolist()
        # every request reads the tokens of its parent
        for r in range(n):
            if p[r] >= 0:
                nb = ref.held(lens[p[r]], block, width)
                assert torch.equal(cache[f.table[r, :nb].long()], before[t[p[r], :nb].long()])


def test_a_beam_search_over_a_shared_cache():
    """Beams select, states reorder, tables fork and grow; every beam's log is its own history, and compaction keeps it."""
    torch.manual_seed(0)
    n, k, vocab, block, blocks, width, steps = 3, 4, 50, 4, 120, 16, 23
    scores = torch.zeros(n, k, device="cuda")
    scores[:, 1:] = -float("inf")
    table, lens = torch.full((n * k, width), -1, dtype=torch.int32, device="cuda"), torch.zeros(n * k, dtype=torch.int32, device="cuda")
    log, state = torch.full((blocks, block), -1, device="cuda"), torch.zeros(n, k, 6, device="cuda")
    history = [[[] for _ in range(k)] for _ in range(n)]
    base = (torch.arange(n, device="cuda", dtype=torch.int32) * k)[:, None]
    gate = torch.full((n * k, 6), -0.1, device="cuda")
    refs = ak.ak_blocks_count(table, lens, block_size=block, blocks=blocks)
    for _ in range(steps):
        logits = torch.randn(n, k, vocab, device="cuda") * 2
        step = ak.ak_beam_select(logits, scores)
        scores = step.scores
        ak.ak_beam_reorder(state, step.parents)
        free, _ = ak.ak_blocks_free(refs)
        f = ak.ak_blocks_fork(table, lens, (base + step.parents).reshape(-1), free, block_size=block, blocks=blocks)
        ak.ak_blocks_copy(log, f.pairs, counts=f.counts)
        free, _ = ak.ak_blocks_free(f.refs)
        one = torch.ones(n * k, dtype=torch.int32, device="cuda")
        lay = ak.ak_batch_layout(f.lens, one, f.table, free, block_size=block, max_tokens=n * k)
        token = step.tokens.reshape(-1)
        log.reshape(-1)[lay.slots] = token.long()
        ak.ak_gated_recurrence_step(token[:, None].float().expand(-1, 6).contiguous(), gate, state.view(n * k, 6))
        table, lens = f.table, f.lens + 1
        refs = ak.ak_blocks_count(table, lens, block_size=block, blocks=blocks)
        history = [[history[r][step.parents[r, j]] + [int(step.tokens[r, j])] for j in range(k)] for r in range(n)]
    for move in range(2):
        for r in range(n):
            for j in range(k):
                row = table[r * k + j, : -(-steps // block)].long()
                assert log[row].reshape(-1)[:steps].tolist() == history[r][j]
                want = 0.0
                for t in history[r][j]:
                    want = np.exp(np.float32(-0.1).astype(np.float64)) * want + t
                # 23 steps of three roundings each
                assert abs(float(state[r, j, 0]) - want) <= 3 * steps * 2.0**-24 * want
        if not move:
            table, pairs, counts = ak.ak_blocks_compact(table, lens, refs, block_size=block)
            ak.ak_blocks_copy(log, pairs, counts=counts)
            refs = ak.ak_blocks_count(table, lens, block_size=block, blocks=blocks)
            used = int(counts[1])
            assert (refs[:used] > 0).all() and not refs[used:].any()
