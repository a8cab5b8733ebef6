"""Cases and plain forms of further sequence operators: a gated linear recurrence over packed sequences (its gradients, its single
tokens), beam search's selection with the reordering of states, and the forking, copying, freeing and compacting of a paged cache's
blocks.

`run` computes a case in elementary torch operations, or with `own` through the package's entry points.
"""
import math

import numpy as np
import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# --------------------------------------------------------------------------------------------------------------- cases


def listed():
    return [
        # a serving batch of ragged prompts
        dict(name="recur_packed", op="recur", form="decay", dtype="bf16", tokens=16384, seqs=16, channels=4096, state=False, final=True),
        # drafted tokens of many requests taken into their states at once, a width off the powers of two
        dict(name="recur_drafts", op="recur", form="gate", dtype="f32", tokens=331, seqs=64, channels=1000, state=True, final=True),
        # a training step's forward and backward, packed documents
        dict(name="train_packed", op="train", form="gate", dtype="bf16", tokens=8192, seqs=5, channels=4096, state=False, final=False),
        # one long document by segments: few channels, a long axis, the state and its gradient cross the segment's ends
        dict(name="train_long", op="train", form="decay", dtype="f32", tokens=32771, seqs=1, channels=640, state=True, final=True),
        # one token for each request of a full decode batch
        dict(name="step_batch", op="step", form="gate", dtype="bf16", batch=256, channels=4096),
        # one token of a single user
        dict(name="step_one", op="step", form="decay", dtype="bf16", batch=1, channels=2560),
        # a few beams of one user, a mid-sized vocabulary of odd size
        dict(name="beam_few", op="beam", dtype="f32", batch=1, beams=4, vocab=32003, layers=4, width=1024, penalty=1.0),
        # a full batch, a large vocabulary
        dict(name="beam_batch", op="beam", dtype="bf16", batch=64, beams=8, vocab=128000, layers=8, width=2048, penalty=0.6),
        # the beams of two users fork their cache
        dict(name="fork_few", op="fork", groups=2, beams=4, ctx=600, block=16, heads=2, dim=64, layers=2),
        # a full batch's beams
        dict(name="fork_batch", op="fork", groups=64, beams=8, ctx=4000, block=16, heads=4, dim=64, layers=2),
        # a small pool after some requests have left
        dict(name="compact_few", op="compact", seqs=16, ctx=300, block=16, heads=2, dim=64, layers=2),
        # a large one
        dict(name="compact_batch", op="compact", seqs=256, ctx=4000, block=16, heads=4, dim=64, layers=1),
    ]


def _span(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["recur", "recur", "train", "step", "beam", "beam", "fork", "compact"])
    if op in ("recur", "train"):
        dtype = rng.choice(["bf16", "bf16", "f32"])
        channels = _span(rng, 200, 8192)
        if rng.random() < 0.75:
            channels = -(-channels // 8) * 8
        most = (6e7 if op == "recur" else 3e7) / (1 if dtype == "bf16" else 2)
        tokens = _span(rng, 40, min(32771, most / channels))
        return dict(op=op, form=rng.choice(["decay", "gate"]), dtype=dtype, tokens=tokens, seqs=_span(rng, 1, max(1, min(64, tokens // 8))),
                    channels=channels, state=rng.random() < 0.5, final=rng.random() < 0.6)
    if op == "step":
        return dict(op=op, form=rng.choice(["decay", "gate"]), dtype=rng.choice(["bf16", "bf16", "f32"]), batch=_span(rng, 1, 256),
                    channels=rng.choice([640, 1000, 1536, 2048, 2560, 4096]))
    if op == "beam":
        beams = rng.choice([1, 2, 4, 5, 8, 16])
        dtype = rng.choice(["bf16", "f32"])
        vocab = _span(rng, 1000, 128000)
        most = 6e7 / (1 if dtype == "bf16" else 2) / (beams * vocab)
        return dict(op=op, dtype=dtype, batch=_span(rng, 1, max(1, min(64, most))), beams=beams, vocab=vocab, layers=rng.randint(1, 8),
                    width=rng.choice([64, 500, 1024, 2048]), penalty=rng.choice([0.0, 0.6, 1.0]))
    block, heads, dim = rng.choice([8, 16, 24, 32]), rng.choice([1, 2, 4]), rng.choice([64, 80, 128])
    ctx, layers = _span(rng, 20, 4000), rng.randint(1, 3)
    page = block * heads * dim * 2 * layers
    if op == "fork":
        beams = rng.choice([2, 4, 5, 8, 16])
        one = (-(-ctx // block) + 1) * (0.7 + 0.3 * beams) * page  # bytes of a group's blocks
        return dict(op=op, groups=_span(rng, 1, max(1, min(64, 7e8 / one))), beams=beams, ctx=ctx, block=block, heads=heads, dim=dim, layers=layers)
    one = -(-ctx // block) * page
    return dict(op=op, seqs=_span(rng, 4, max(4, min(256, 4e8 / one))), ctx=ctx, block=block, heads=heads, dim=dim, layers=layers)


def _fork_pool(case):
    """Blocks of a fork case's pool: at most 0.3 of a request's blocks are its own, and every request may take one more."""
    nb = -(-case["ctx"] // case["block"])
    return case["groups"] * (nb + case["beams"] * (math.ceil(0.3 * nb) + 1)) + 8


def work(case):
    op = case["op"]
    if op in ("recur", "train"):
        e = 2 if case["dtype"] == "bf16" else 4
        n = case["tokens"] * case["channels"]
        states = case["seqs"] * case["channels"] * 4 * (case["state"] + case["final"])
        if op == "recur":
            return {"bytes": 3 * n * e + states, "flops": 3 * n}
        # the backward pass reads gate, dh and h (or x) and writes dx and dgate (and the states' gradients)
        return {"bytes": 8 * n * e + 2 * states, "flops": 10 * n}
    if op == "step":
        e = 2 if case["dtype"] == "bf16" else 4
        n = case["batch"] * case["channels"]
        return {"bytes": 8 * n + 3 * n * e, "flops": 3 * n}
    if op == "beam":
        e = 2 if case["dtype"] == "bf16" else 4
        n = case["batch"] * case["beams"] * case["vocab"] * 0.85  # finished beams' rows are not needed
        moved = case["batch"] * case["layers"] * case["width"] * 4 * (case["beams"] - 1)
        return {"bytes": n * e + 1.5 * moved, "flops": 4 * n}
    page = case["block"] * case["heads"] * case["dim"] * 2 * case["layers"]
    if op == "fork":
        rows = case["groups"] * case["beams"]
        entries = rows * 0.75 * case["ctx"] / case["block"]
        return {"bytes": 8 * entries + 8 * _fork_pool(case) + 0.35 * rows * 2 * page, "flops": entries}
    entries = case["seqs"] * 0.5 * case["ctx"] / case["block"]
    return {"bytes": 8 * entries + 4 * case["seqs"] * -(-case["ctx"] // case["block"]) + 0.5 * entries * 2 * page, "flops": entries}


# -------------------------------------------------------------------------------------------------------------- inputs


def _lengths(total, seqs, rng):
    """`seqs` lengths that sum to `total`, spread about their mean; with eight or more, one of them 0 and one 1."""
    w = rng.uniform(0.25, 1.75, seqs)
    special = seqs >= 8 and total >= 4 * seqs
    if special:
        w[[2, 5]] = 0
    n = np.floor(w / w.sum() * (total - special)).astype(np.int64)
    if special:
        n[5] = 1
    n[int(np.argmax(w))] += total - n.sum()
    return n


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    rng = np.random.default_rng(seed)
    s = dict(case)

    def normal(*shape, dtype=torch.float32, scale=1.0):
        return (torch.randn(*shape, generator=g, device=dev, dtype=torch.float32) * scale).to(dtype)

    def gates(rows, channels, form, dtype):
        # channels of every memory, from a token to thousands; a token's gate varies about its channel's
        c = torch.rand(channels, generator=g, device=dev)
        z = normal(rows, channels)
        if form == "decay":
            return (-torch.exp(z.add_(c * 9 - 8))).to(dtype)  # a log decay, -1e-4 to -10
        return z.mul_(1.5).add_(c * 8 - 2).to(dtype)  # a logit

    def ints(x):
        return torch.tensor(np.asarray(x), dtype=torch.int32, device=dev)

    op = case["op"]
    if op in ("recur", "train"):
        t, n, c, dt = case["tokens"], case["seqs"], case["channels"], TYPES[case["dtype"]]
        s["lens"] = _lengths(t, n, rng)
        s["offsets"] = ints(np.concatenate([[0], np.cumsum(s["lens"])]))
        s["gate"] = gates(t, c, case["form"], dt)
        s["x"] = normal(t, c, dtype=dt)
        s["s0"] = normal(n, c) if case["state"] else None
        if op == "train":
            s["dh"] = normal(t, c, dtype=dt)
            s["ds"] = normal(n, c) if case["final"] else None
    elif op == "step":
        b, c, dt = case["batch"], case["channels"], TYPES[case["dtype"]]
        s["gate"], s["x"] = gates(b, c, case["form"], dt), normal(b, c, dtype=dt)
        pool = b + b // 4 + 1
        s["pool"] = normal(pool, c)
        s["slots"] = ints(rng.permutation(pool)[:b])
    elif op == "beam":
        b, k, v, dt = case["batch"], case["beams"], case["vocab"], TYPES[case["dtype"]]
        s["logits"] = normal(b, k, v, dtype=dt, scale=2.5)
        s["scores"] = -torch.rand(b, k, generator=g, device=dev) * 3 - 10
        # a beam in seven has ended; the first of a request goes on
        done = torch.rand(b, k, generator=g, device=dev) < 0.15
        done[:, 0] = False
        s["done"] = done
        s["lengths"] = torch.where(done, ints(rng.integers(8, 21, (b, k))), 20).int()
        s["end"] = min(2, v - 1)
        s["state"] = normal(case["layers"], b, k, case["width"])
    elif op == "fork":
        n, k, block = case["groups"], case["beams"], case["block"]
        pool = _fork_pool(case)
        ids = rng.permutation(pool)
        width = -(-case["ctx"] // block) + 2
        table = np.full((n * k, width), -1, np.int32)
        lens, parents, at = np.zeros(n * k, np.int32), np.zeros(n * k, np.int32), 0
        for i in range(n):  # beams share their prefix's blocks and have the last ones to themselves
            length = int(rng.integers(case["ctx"] // 2, case["ctx"] + 1))
            nb = -(-length // block)
            alone = max(1, int(rng.uniform(0.02, 0.3) * nb))
            rows = slice(i * k, i * k + k)
            lens[rows] = length
            table[rows, : nb - alone] = ids[at: at + nb - alone]
            at += nb - alone
            table[rows, nb - alone: nb] = ids[at: at + k * alone].reshape(k, alone)
            at += k * alone
            parents[rows] = i * k + rng.integers(0, k, k)
            if n > 4 and rng.random() < 0.08:
                parents[rows] = -1  # a request that has ended
        s["table"], s["lens"], s["parents"], s["free"], s["blocks"] = ints(table), ints(lens), ints(parents), ints(ids[at:]), pool
    else:
        n, block = case["seqs"], case["block"]
        width = -(-case["ctx"] // block)
        pool = n * width
        ids = rng.permutation(pool)
        lens = rng.integers(0, case["ctx"] + 1, n)
        table = np.full((n, width), -1, np.int32)
        at = 0
        for i in range(n):
            nb = -(-int(lens[i]) // block)
            table[i, :nb] = ids[at: at + nb]
            if i % 5 == 4:  # a prefix shared with the request before
                same = min(nb, -(-int(lens[i - 1]) // block)) // 2
                table[i, :same] = table[i - 1, :same]
            at += nb
        s["table"], s["lens"], s["blocks"] = ints(table), ints(lens), pool
    if op in ("fork", "compact"):
        s["cache"] = normal(case["layers"], pool, case["block"], case["heads"], case["dim"], dtype=torch.bfloat16)
    return s


# --------------------------------------------------------------------------------------------------------- plain forms


def _weights(gate, form):
    """a, a - 1 and b of h_t = a_t h_{t-1} + b_t x_t: a long memory's a says little about its distance from 1."""
    g = gate.float()
    if form == "decay":
        return torch.exp(g), torch.expm1(g), None
    e = torch.exp(-g.abs())
    r = 1 / (1 + e)
    b = torch.where(g >= 0, e * r, r)
    return torch.where(g >= 0, r, e * r), -b, b


def _scan(m, u, first, longest):
    """y_t = (1 + m_t) y_{t-1} + u_t down the rows, from 0 at the rows `first`, by doubling. m and u are overwritten."""
    starts = torch.zeros(u.shape[0], 1, dtype=torch.bool, device=u.device)
    starts[first] = True
    d = 1
    while d < longest:
        u[d:] += torch.where(starts[d:], 0, u[:-d] + m[d:] * u[:-d])
        m[d:] = m[d:] + m[:-d] + m[d:] * m[:-d]
        starts[d:] = starts[d:] | starts[:-d]
        d *= 2
    return u


def _plain_forward(s):
    """h (float32) and the states after each sequence."""
    off, s0, longest = s["offsets"].long(), s["s0"], int(s["lens"].max())
    some = off[1:] > off[:-1]
    first, last = off[:-1][some], off[1:][some] - 1
    a, m, b = _weights(s["gate"], s["form"])
    u = s["x"].float() if b is None else b * s["x"].float()
    if s0 is not None:
        u[first] += a[first] * s0[some]
    h = _scan(m, u, first, longest)
    if not s["final"]:
        return h, None
    sf = torch.zeros(s["seqs"], h.shape[1], device=h.device) if s0 is None else s0.clone()
    sf[some] = h[last]
    return h, sf


def _plain_backward(s, h):
    off, s0, ds, longest = s["offsets"].long(), s["s0"], s["ds"], int(s["lens"].max())
    some = off[1:] > off[:-1]
    first, last = off[:-1][some], off[1:][some] - 1
    a, m, b = _weights(s["gate"], s["form"])
    # time backwards: G_t = dh_t + a_{t+1} G_{t+1}
    u = s["dh"].float().flip(0)
    w = torch.zeros_like(m)
    w[1:] = m.flip(0)[:-1]
    del m
    rev_last = h.shape[0] - 1 - last
    if ds is not None:
        u[rev_last] += ds[some]
    gr = _scan(w, u, rev_last, longest).flip(0)
    del w, u
    before = torch.zeros_like(h)
    before[1:] = h[:-1]
    before[first] = 0 if s0 is None else s0[some]
    if b is None:
        dx, dg = gr, gr * a * before
    else:
        dx, dg = gr * b, gr * (before - s["x"].float()) * a * b
    d0 = None
    if s0 is not None:
        d0 = torch.zeros_like(s0) if ds is None else ds.clone()
        d0[some] = a[first] * gr[first]
    dt = s["x"].dtype
    return dx.to(dt), dg.to(dt), d0


def _plain_step(s):
    at = s["slots"].long()
    a, _, b = _weights(s["gate"], s["form"])
    x = s["x"].float()
    h = a * s["pool"][at] + (x if b is None else b * x)
    s["pool"][at] = h
    return h.to(s["x"].dtype)


def _plain_select(s):
    """Scores next to one another decide: sums of logits and the comparisons are in 64 bits."""
    x, score, done, length = s["logits"].double(), s["scores"].double(), s["done"], s["lengths"]
    b, k, v = x.shape
    dev = x.device
    m = x.amax(-1, keepdim=True)
    total = x - (m + torch.exp(x - m).sum(-1, keepdim=True).log()) + score[..., None]
    new = length + (~done).int()
    col = torch.arange(v, device=dev)
    total = torch.where(done[..., None], torch.where(col == s["end"], score[..., None], -math.inf), total)
    rank = (total / (new.double() ** s["penalty"])[..., None]).reshape(b, k * v)
    total = total.reshape(b, k * v)
    flat = torch.arange(k * v, device=dev)
    picks = []
    for _ in range(k):
        best = rank.amax(1, keepdim=True)
        at = torch.where(rank == best, flat, k * v).amin(1, keepdim=True)
        picks.append(at)
        rank.scatter_(1, at, -math.inf)
    at = torch.cat(picks, 1)
    parents, tokens = at // v, at % v
    ended = done.gather(1, parents) | (tokens == s["end"])
    return total.gather(1, at).float(), tokens.int(), parents.int(), ended, new.gather(1, parents)


def _plain_reorder(state, parents):
    layers, b, k, w = state.shape
    state.copy_(state.gather(2, parents.long()[None, :, :, None].expand(layers, b, k, w)))


def _used(table, lens, block):
    """Which entries of a table hold a request's blocks."""
    return torch.arange(table.shape[1], device=table.device)[None] < ((lens + block - 1) // block)[:, None]


def _plain_count(table, lens, block, blocks):
    held = table[_used(table, lens, block)].long()
    return torch.zeros(blocks, dtype=torch.int32, device=table.device).index_add_(0, held, torch.ones_like(held, dtype=torch.int32))


def _listed_first(ids, size):
    """ids, then -1 up to `size` of them."""
    out = torch.full((size,) + ids.shape[1:], -1, dtype=torch.int32, device=ids.device)
    out[: ids.shape[0]] = ids
    return out


def _plain_copy(cache, pairs):
    cache[:, pairs[:, 1].long()] = cache[:, pairs[:, 0].long()]


def _plain_fork(s):
    parents, block, blocks = s["parents"].long(), s["block"], s["blocks"]
    n, width = s["table"].shape
    dev = parents.device
    live = parents >= 0
    at = parents.clamp(min=0)
    lens = torch.where(live, s["lens"][at], 0)
    table = torch.where(_used(s["table"], lens, block), s["table"][at], -1)
    refs = _plain_count(table, lens, block, blocks)
    # a partly filled last block may be written next: one of those that end in it keeps it, if nobody else holds it
    rows = torch.arange(n, device=dev)
    col = lens.long() // block
    partial = live & (lens % block != 0)
    tail = torch.where(partial, table[rows, col.clamp(max=width - 1)].long(), blocks)
    one = torch.ones_like(tail, dtype=torch.int32)
    ends = torch.zeros(blocks + 1, dtype=torch.int32, device=dev).index_add_(0, tail, one)
    keeper = torch.full((blocks + 1,), n, device=dev).scatter_reduce_(0, tail, rows, "amin")
    all_refs = torch.cat([refs, refs[:1]])
    copy = partial & ~((keeper[tail] == rows) & (all_refs[tail] <= ends[tail]))
    r = rows[copy]
    src = tail[copy]
    dst = s["free"][: r.numel()].long()
    table[r, col[copy]] = dst.int()
    refs.index_add_(0, src, -torch.ones_like(src, dtype=torch.int32))
    refs[dst] = 1
    pairs = torch.stack([src, dst], 1).int()
    _plain_copy(s["cache"], pairs)
    free = torch.nonzero(refs == 0)[:, 0].int()
    return {"table": table, "lens": lens, "refs": refs, "pairs": _listed_first(pairs, n), "counts": copy.sum()[None].int(),
            "free": _listed_first(free, blocks), "nfree": torch.tensor([free.numel()], dtype=torch.int32, device=dev), "cache": s["cache"]}


def _plain_compact(s):
    block, blocks = s["block"], s["blocks"]
    refs = _plain_count(s["table"], s["lens"], block, blocks)
    live = refs > 0
    n = int(live.sum())
    src = torch.nonzero(live[n:])[:, 0] + n
    dst = torch.nonzero(~live[:n])[:, 0]
    to = torch.arange(blocks, device=live.device)
    to[src] = dst
    table = torch.where(_used(s["table"], s["lens"], block), to[s["table"].clamp(min=0).long()].int(), s["table"])
    pairs = torch.stack([src, dst], 1).int()
    _plain_copy(s["cache"], pairs)
    return {"refs": refs, "table": table, "pairs": _listed_first(pairs, blocks // 2),
            "counts": torch.tensor([src.numel(), n], dtype=torch.int32, device=live.device), "cache": s["cache"]}


# ----------------------------------------------------------------------------------------------------------------- run


def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_plain(s):
    op = s["op"]
    if op in ("recur", "train"):
        h, sf = _plain_forward(s)
        out = {"h": h.to(s["x"].dtype), "state": sf}
        if op == "train":
            out["dx"], out["dgate"], out["dstate"] = _plain_backward(s, h)
        return out
    if op == "step":
        return {"h": _plain_step(s), "pool": s["pool"]}
    if op == "beam":
        scores, tokens, parents, done, lengths = _plain_select(s)
        _plain_reorder(s["state"], parents)
        return {"scores": scores, "tokens": tokens, "parents": parents, "done": done, "lengths": lengths, "state": s["state"]}
    return _plain_fork(s) if op == "fork" else _plain_compact(s)


def _run_own(s):
    import mapreduce_prefix_scan_gb300 as ak

    op = s["op"]
    if op in ("recur", "train"):
        same = dict(form=s["form"], offsets=s["offsets"], state=s["s0"])
        # the plain form's scan is in x's own memory where x needs no conversion and no factor, and so is the call
        place = s["x"] if s["dtype"] == "f32" and s["form"] == "decay" else None
        h, sf = ak.ak_gated_recurrence(s["x"], s["gate"], out=place, final_state=s["final"], **same)
        if op == "recur":
            return {"h": h, "state": sf}
        dx, dgate, d0 = ak.ak_gated_recurrence_backward(s["dh"], s["x"], s["gate"], h, dstate_out=s["ds"], **same)
        return {"h": h, "state": sf, "dx": dx, "dgate": dgate, "dstate": d0}
    if op == "step":
        h = ak.ak_gated_recurrence_step(s["x"], s["gate"], s["pool"], slots=s["slots"], form=s["form"])
        return {"h": h, "pool": s["pool"]}
    if op == "beam":
        r = ak.ak_beam_select(s["logits"], s["scores"], done=s["done"], lengths=s["lengths"], end_token=s["end"], length_penalty=s["penalty"])
        ak.ak_beam_reorder(s["state"], r.parents, dim=1)
        return {"scores": r.scores, "tokens": r.tokens, "parents": r.parents, "done": r.done, "lengths": r.lengths, "state": s["state"]}
    if op == "fork":
        f = ak.ak_blocks_fork(s["table"], s["lens"], s["parents"], s["free"], block_size=s["block"], blocks=s["blocks"])
        ak.ak_blocks_copy(s["cache"], f.pairs, counts=f.counts, dim=1)
        free, nfree = ak.ak_blocks_free(f.refs)
        return {"table": f.table, "lens": f.lens, "refs": f.refs, "pairs": f.pairs, "counts": f.counts, "free": free, "nfree": nfree,
                "cache": s["cache"]}
    refs = ak.ak_blocks_count(s["table"], s["lens"], block_size=s["block"], blocks=s["blocks"])
    table, pairs, counts = ak.ak_blocks_compact(s["table"], s["lens"], refs, block_size=s["block"])
    ak.ak_blocks_copy(s["cache"], pairs, counts=counts, dim=1)
    return {"refs": refs, "table": table, "pairs": pairs, "counts": counts, "cache": s["cache"]}


# --------------------------------------------------------------------------------------------------------------- exact


def exact(case, seed):
    s = prepare(case, seed)
    with torch.no_grad():
        if case["op"] in ("recur", "train"):
            return _exact_recurrence(s, case["op"] == "train")
        if case["op"] == "step":
            return _exact_step(s)
        if case["op"] == "beam":
            return _exact_beam(s)
        return _exact_fork(s) if case["op"] == "fork" else _exact_compact(s)


def _exact_weights(gate, form):
    g = gate.double()
    return (g.exp(), torch.ones_like(g)) if form == "decay" else (g.sigmoid(), (-g).sigmoid())


def _exact_recurrence(s, train):
    """Token by token from the recurrences, all sequences side by side, the longest first."""
    lens = s["lens"]
    order = np.argsort(-lens, kind="stable")
    starts = np.concatenate([[0], np.cumsum(lens)[:-1]])[order]
    dev = s["x"].device
    starts = torch.as_tensor(starts, device=dev)
    order_t, back = torch.as_tensor(order, device=dev), torch.as_tensor(np.argsort(order), device=dev)
    ends = starts + torch.as_tensor(lens[order], device=dev) - 1
    live = [int((lens > i).sum()) for i in range(int(lens.max()))]
    a, b = _exact_weights(s["gate"], s["form"])
    x = s["x"].double()
    h = torch.zeros_like(x)
    S = torch.zeros(len(lens), x.shape[1], dtype=torch.float64, device=dev)
    if s["s0"] is not None:
        S = s["s0"].double()[order_t].clone()
    u = b * x
    before = torch.zeros_like(x) if train else None
    for i, m in enumerate(live):
        at = starts[:m] + i
        if train:
            before[at] = S[:m]
        S[:m] = a[at] * S[:m] + u[at]
        h[at] = S[:m]
    out = {"h": h, "state": S[back] if s["final"] else None}
    if train:
        del u
        G = torch.zeros_like(S) if s["ds"] is None else s["ds"].double()[order_t].clone()
        gr = torch.zeros_like(x)
        dh = s["dh"].double()
        for i, m in enumerate(live):
            at = ends[:m] - i
            G[:m] += dh[at]
            gr[at] = G[:m]
            G[:m] *= a[at]
        da = before if s["form"] == "decay" else before - x
        out |= {"dx": gr * b, "dgate": gr * da * a * (1 if s["form"] == "decay" else b), "dstate": G[back] if s["s0"] is not None else None}
    return out


def _exact_step(s):
    pool = s["pool"].double()
    a, b = _exact_weights(s["gate"], s["form"])
    h = torch.zeros_like(a)
    for i, slot in enumerate(s["slots"].tolist()):
        pool[slot] = a[i] * pool[slot] + b[i] * s["x"][i].double()
        h[i] = pool[slot]
    return {"h": h, "pool": pool}


def _exact_beam(s):
    b, k, v = s["logits"].shape
    out = {"scores": torch.zeros(b, k, dtype=torch.float64), "tokens": torch.zeros(b, k, dtype=torch.int32), "parents": torch.zeros(b, k, dtype=torch.int32),
           "done": torch.zeros(b, k, dtype=torch.bool), "lengths": torch.zeros(b, k, dtype=torch.int32)}
    scores, done, lengths = s["scores"].double().tolist(), s["done"].tolist(), s["lengths"].tolist()
    state = s["state"].clone()
    for i in range(b):
        logp = torch.log_softmax(s["logits"][i].double(), -1)
        picks = []
        for j in range(k):
            if done[i][j]:
                picks.append((-scores[i][j] / lengths[i][j] ** s["penalty"], j, s["end"], scores[i][j]))
                continue
            val, tok = torch.sort(logp[j], descending=True, stable=True)
            for x, t in zip(val[:k].tolist(), tok[:k].tolist()):
                picks.append((-(scores[i][j] + x) / (lengths[i][j] + 1) ** s["penalty"], j, t, scores[i][j] + x))
        for q, (_, j, t, total) in enumerate(sorted(picks)[:k]):
            out["scores"][i, q], out["tokens"][i, q], out["parents"][i, q] = total, t, j
            out["done"][i, q] = done[i][j] or t == s["end"]
            out["lengths"][i, q] = lengths[i][j] + (not done[i][j])
            state[:, i, q] = s["state"][:, i, j]
    return out | {"state": state}


def _numpy(s, *names):
    return [s[x].cpu().numpy().astype(np.int64) for x in names]


def _padded(rows, shape):
    out = np.full(shape, -1, np.int32)
    if rows:
        out[: len(rows)] = rows
    return out


def _exact_fork(s):
    table, lens, parents, free = _numpy(s, "table", "lens", "parents", "free")
    b, blocks, n = s["block"], s["blocks"], len(parents)
    new, new_lens, refs = np.full_like(table, -1), np.zeros(n, np.int64), np.zeros(blocks, np.int64)
    ends = {}
    for r, p in enumerate(parents):
        if p < 0:
            continue
        new_lens[r] = lens[p]
        nb = -(-int(lens[p]) // b)
        new[r, :nb] = table[p, :nb]
        refs[new[r, :nb]] += 1  # a request's blocks are distinct
        if lens[p] % b:
            ends.setdefault(int(new[r, nb - 1]), []).append(r)
    copies = sorted(r for block, rows in ends.items() for r in (rows[1:] if refs[block] <= len(rows) else rows))
    pairs = []
    for r, dst in zip(copies, free):
        col = int(new_lens[r]) // b
        pairs.append((int(new[r, col]), int(dst)))
        refs[new[r, col]] -= 1
        new[r, col], refs[dst] = dst, 1
    cache = s["cache"]
    for src, dst in pairs:
        cache[:, dst] = cache[:, src]
    left = np.flatnonzero(refs == 0)
    return {"table": new.astype(np.int32), "lens": new_lens.astype(np.int32), "refs": refs.astype(np.int32), "pairs": _padded(pairs, (n, 2)),
            "counts": np.array([len(pairs)], np.int32), "free": _padded(list(left), blocks), "nfree": np.array([len(left)], np.int32), "cache": cache}


def _exact_compact(s):
    table, lens = _numpy(s, "table", "lens")
    b, blocks, cache = s["block"], s["blocks"], s["cache"]
    refs = np.zeros(blocks, np.int64)
    held = [-(-int(m) // b) for m in lens]
    for r, nb in enumerate(held):
        refs[table[r, :nb]] += 1
    used = [i for i in range(blocks) if refs[i] > 0]
    n = len(used)
    holes = [i for i in range(n) if refs[i] == 0]
    pairs = list(zip([i for i in used if i >= n], holes))
    to = dict(pairs)
    for r, nb in enumerate(held):
        table[r, :nb] = [to.get(int(i), int(i)) for i in table[r, :nb]]
    if pairs:
        src, dst = (torch.tensor(x, device=cache.device) for x in zip(*pairs))
        cache[:, dst] = cache[:, src]
    return {"refs": refs.astype(np.int32), "table": table.astype(np.int32), "pairs": _padded(pairs, (blocks // 2, 2)),
            "counts": np.array([len(pairs), n], np.int32), "cache": cache}
