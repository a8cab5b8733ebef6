"""Cases and plain forms of the sequence operators: linear attention with a decay for each head (packed prompts, its gradients,
single tokens), the layout of a batch from its request lengths, and the verification of drafted tokens.

`run` computes a case in elementary torch operations, or with `own` through the package's entry points.
"""
import math

import numpy as np
import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
CHUNK = 64


# --------------------------------------------------------------------------------------------------------------- cases


def listed():
    return [
        # a serving batch of ragged prompts behind one packed qkv projection
        dict(name="prompt_packed", op="prompt", dtype="bf16", tokens=16384, seqs=16, heads=32, dim=128, state=False, final=True),
        # one long document: few rows, a long axis
        dict(name="prompt_long", op="prompt", dtype="bf16", tokens=32771, seqs=1, heads=16, dim=128, state=False, final=True),
        # drafted tokens of many requests taken into their states at once (a few tokens each)
        dict(name="prompt_drafts", op="prompt", dtype="bf16", tokens=331, seqs=64, heads=16, dim=64, state=True, final=True),
        # the same operator in 32 bits, a head size off the powers of two
        dict(name="prompt_f32", op="prompt", dtype="f32", tokens=2049, seqs=5, heads=8, dim=80, state=True, final=True),
        # a training step's forward and backward, packed documents
        dict(name="train_packed", op="train", dtype="bf16", tokens=8192, seqs=4, heads=16, dim=128, state=False, final=False),
        # training by segments: the state and its gradient cross the segment's ends
        dict(name="train_segment", op="train", dtype="bf16", tokens=1000, seqs=2, heads=12, dim=64, state=True, final=True),
        # one token for each request of a full decode batch
        dict(name="step_batch", op="step", dtype="bf16", batch=256, heads=32, dim=128),
        # one token of a single user
        dict(name="step_one", op="step", dtype="bf16", batch=1, heads=16, dim=128),
        # the batch of a decode step: one new token a request
        dict(name="layout_decode", op="layout", seqs=256, tokens=256, block=16, ctx=4000, width=512),
        # prompts and decodes mixed, a large batch
        dict(name="layout_mixed", op="layout", seqs=2047, tokens=1000003, block=16, ctx=3000, width=640),
        # a few requests, a mid-sized vocabulary of odd size
        dict(name="verify_few", op="verify", dtype="f32", seqs=4, drafts=3, vocab=32003, drafted=True),
        # a full batch, a large vocabulary
        dict(name="verify_batch", op="verify", dtype="f32", seqs=192, drafts=5, vocab=128000, drafted=True),
    ]


def _span(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["prompt", "prompt", "train", "step", "layout", "verify"])
    if op in ("prompt", "train"):
        dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
        dim = rng.choice([64, 128]) if dtype == "bf16" else rng.choice([32, 64, 80, 128])
        heads = rng.choice([4, 7, 8, 12, 16, 32])
        most = (6e6 if op == "prompt" else 2e6) / (1 if dtype == "bf16" else 8)
        tokens = _span(rng, 60, max(200, most / (heads * dim) * 8))
        seqs = _span(rng, 1, max(1, min(64, tokens // 8)))
        return dict(op=op, dtype=dtype, tokens=tokens, seqs=seqs, heads=heads, dim=dim, state=rng.random() < 0.5, final=rng.random() < 0.7)
    if op == "step":
        return dict(op=op, dtype=rng.choice(["bf16", "bf16", "f32"]), batch=_span(rng, 1, 256), heads=rng.choice([4, 7, 8, 16, 32]), dim=rng.choice([64, 80, 128]))
    if op == "layout":
        seqs = _span(rng, 1, 4096)
        return dict(op=op, seqs=seqs, tokens=_span(rng, seqs, max(seqs * 2, 800000)), block=rng.choice([8, 16, 24, 32, 64]), ctx=_span(rng, 16, 3000), width=1024)
    return dict(op=op, dtype=rng.choice(["f32", "f32", "bf16"]), seqs=_span(rng, 1, 160), drafts=rng.randint(1, 6), vocab=_span(rng, 1000, 128000), drafted=rng.random() < 0.75)


def work(case):
    if case["op"] in ("prompt", "train"):
        e = 2 if case["dtype"] == "bf16" else 4
        rows = case["tokens"] * case["heads"] * case["dim"]
        states = case["seqs"] * case["heads"] * case["dim"] ** 2 * 4 * (case["state"] + case["final"])
        flops = 4 * rows * case["dim"]
        if case["op"] == "prompt":
            return {"bytes": 4 * rows * e + states, "flops": flops}
        # the backward pass reads q, k, v and do and writes dq, dk, dv (and the states' gradients)
        return {"bytes": 11 * rows * e + 2 * states + case["seqs"] * case["heads"] * case["dim"] ** 2 * 4 * case["state"], "flops": 4 * flops}
    if case["op"] == "step":
        e = 2 if case["dtype"] == "bf16" else 4
        rows = case["batch"] * case["heads"] * case["dim"]
        return {"bytes": 8 * rows * case["dim"] + 4 * rows * e, "flops": 4 * rows * case["dim"]}
    if case["op"] == "layout":
        blocks = case["tokens"] / case["block"] + case["seqs"] * 0.5
        return {"bytes": 16 * case["tokens"] + 12 * case["seqs"] + 8 * blocks, "flops": 8 * case["tokens"]}
    e = 2 if case["dtype"] == "bf16" else 4
    refused = 1 - 0.75 ** case["drafts"] if case["drafted"] else 1  # the bonus row of a request has no draft row
    n = case["seqs"] * case["vocab"]
    return {"bytes": n * (e + 4) + n * e * refused * case["drafted"], "flops": n * 3}


# -------------------------------------------------------------------------------------------------------------- inputs


def _lengths(total, seqs, rng, least=0):
    """`seqs` lengths that sum to `total`, spread about their mean; with eight or more, one of them `least` and one 1."""
    w = rng.uniform(0.25, 1.75, seqs)
    special = seqs >= 8 and total >= 4 * seqs
    if special:
        w[[2, 5]] = 0
    spare = total - (1 + least if special else 0)
    n = np.floor(w / w.sum() * spare).astype(np.int64)
    if special:
        n[2], n[5] = least, 1
    n[int(np.argmax(w))] += total - n.sum()
    if least:
        for i in np.flatnonzero(n < least):
            n[i] += 1
            n[int(np.argmax(n))] -= 1
    return n


def _decays(heads, dev):
    """log of a decay for each head: -2^(-8 (h + 1) / heads)."""
    h = torch.arange(1, heads + 1, device=dev, dtype=torch.float64)
    return (-torch.exp2(-8 * h / heads)).float()


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    rng = np.random.default_rng(seed)
    s = dict(case)

    def normal(*shape, dtype=torch.float32):
        return torch.randn(*shape, generator=g, device=dev, dtype=torch.float32).to(dtype)

    if case["op"] in ("prompt", "train"):
        t, n, h, d = case["tokens"], case["seqs"], case["heads"], case["dim"]
        dt = TYPES[case["dtype"]]
        lens = _lengths(t, n, rng)
        s["lens"] = lens
        s["max_len"] = int(lens.max())
        s["offsets"] = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device=dev)
        qkv = normal(t, 3, h, d, dtype=dt)
        s["q"], s["k"], s["v"] = qkv[:, 0], qkv[:, 1], qkv[:, 2]
        s["log_decay"] = _decays(h, dev)
        s["scale"] = float(np.float32(d ** -0.5))
        s["s0"] = normal(n, h, d, d) if case["state"] else None
        if case["op"] == "train":
            s["do"] = normal(t, h, d, dtype=dt)
            s["ds"] = normal(n, h, d, d) if case["final"] else None
        return s
    if case["op"] == "step":
        b, h, d = case["batch"], case["heads"], case["dim"]
        dt = TYPES[case["dtype"]]
        qkv = normal(b, 3, h, d, dtype=dt)
        s["q"], s["k"], s["v"] = qkv[:, 0], qkv[:, 1], qkv[:, 2]
        s["log_decay"] = _decays(h, dev)
        s["scale"] = float(np.float32(d ** -0.5))
        pool = b + b // 4 + 1
        s["pool"] = normal(pool, h, d, d)
        s["slots"] = torch.tensor(rng.permutation(pool)[:b], dtype=torch.int32, device=dev)
        return s
    if case["op"] == "layout":
        n, t, b = case["seqs"], case["tokens"], case["block"]
        new = _lengths(t, n, rng, least=1)
        ctx = rng.integers(0, case["ctx"] + 1, n)
        # a table wide enough for the longest request
        width = max(case["width"], int(-(-(ctx + new) // b).max()))
        have = -(-ctx // b)
        need = int((-(-(ctx + new) // b) - have).sum())
        ids = rng.permutation(int(have.sum()) + need + 100)
        table = np.full((n, width), -1, np.int32)
        at = np.arange(width)[None, :] < have[:, None]
        table[at] = ids[: int(have.sum())]
        s["ctx_lens"] = torch.tensor(ctx, dtype=torch.int32, device=dev)
        s["new_lens"] = torch.tensor(new, dtype=torch.int32, device=dev)
        s["table"] = torch.tensor(table, device=dev)
        s["free"] = torch.tensor(ids[int(have.sum()):], dtype=torch.int32, device=dev)
        s["max_tokens"] = t + 13  # room past the batch's end, as a fixed-size buffer has
        return s
    n, k, v = case["seqs"], case["drafts"], case["vocab"]
    dt = TYPES[case["dtype"]]
    p = torch.randn(n, k + 1, v, generator=g, device=dev)
    # the drafter is near the target: its logits are the target's and some noise
    q = (p[:, :k] * 3 + torch.randn(n, k, v, generator=g, device=dev) * 0.6).softmax(-1)
    drafts = torch.empty(n, k, dtype=torch.int32, device=dev)
    e = torch.empty(n, v, device=dev)
    for j in range(k):
        drafts[:, j] = (q[:, j] / e.exponential_(generator=g)).argmax(-1)
    s["p"] = p.mul_(3).softmax(-1).to(dt)
    del p
    if not case["drafted"]:  # drafts without a distribution: the target's own likely tokens
        drafts = s["p"][:, :k].argmax(-1).int()
    s["q"] = q.to(dt) if case["drafted"] else None
    s["drafts"] = drafts
    s["counts"] = torch.tensor(rng.integers(max(0, k - 1), k + 1, n), dtype=torch.int32, device=dev)
    s["uniform"] = torch.rand(n, k, generator=g, device=dev)
    s["noise"] = e.exponential_(generator=g).clamp_(min=1e-20)
    return s


# --------------------------------------------------------------------------------------------------------- plain forms


def _decayed(q, k, v, ld, offsets, max_len, init, scale, *, reverse=False, inner=1.0, final=False):
    """The decayed scan in chunks, over sequences padded to one length: out_i = scale (w^(i+1) init + sum_{j<=i} inner w^(i-j) k_j v_j^T)^T q_i
    in float32, and the state after the last token. `reverse` runs time backwards; its state is the gradient that reaches the token before
    the first, so a contribution has decayed once more on leaving and `init` once less on entering."""
    n, (t, h, dk), dv, dev = offsets.numel() - 1, q.shape, v.shape[-1], q.device
    shift, c = int(reverse), CHUNK
    nc = max(1, -(-max_len // c))
    start, end = offsets[:-1].long(), offsets[1:].long()
    at = torch.arange(nc * c, device=dev)
    live = at[None, :] < (end - start)[:, None]
    idx = (end[:, None] - 1 - at[None, :] if reverse else start[:, None] + at[None, :]).clamp(0, max(0, t - 1))

    def rows(x):
        return torch.where(live[:, :, None, None], x[idx].float(), 0.0).permute(0, 2, 1, 3).reshape(n, h, nc, c, x.shape[-1])

    q, k, v = rows(q), rows(k), rows(v)
    i = torch.arange(c, device=dev)
    gap = i[:, None] - i[None, :]
    w = torch.where(gap >= 0, torch.exp(ld[:, None, None] * gap.clamp(min=0)), 0.0) * inner
    out = ((q @ k.transpose(-1, -2)) * w[:, None]) @ v
    leave = torch.exp(ld[:, None] * (c - 1 + shift - i)) * inner
    u = (k * leave[:, None, :, None]).transpose(-1, -2) @ v
    cs = torch.arange(nc, device=dev)
    gap = cs[:, None] - 1 - cs[None, :]
    m = torch.where(gap >= 0, torch.exp(ld[:, None, None] * (c * gap).clamp(min=0)), 0.0)
    s = (m @ u.reshape(n, h, nc, dk * dv)).reshape(n, h, nc, dk, dv)
    if init is not None:
        s = s + torch.exp(ld[:, None] * (c * cs))[:, :, None, None] * init[:, :, None]
    out = out + torch.exp(ld[:, None] * (i + 1 - shift))[:, None, :, None] * (q @ s)
    out = (out * scale).reshape(n, h, nc * c, dv)
    seq = torch.searchsorted(offsets[1:].contiguous(), torch.arange(t, device=dev, dtype=torch.int32), right=True)
    pos = torch.arange(t, device=dev) - start[seq]
    if reverse:
        pos = (end - start)[seq] - 1 - pos
    out = out[seq, :, pos]
    if not final:
        return out, None
    length = (end - start)[:, None]
    left = torch.where(live, length - 1 + shift - at[None, :], 0).float()
    wf = torch.where(live[:, None], torch.exp(ld[None, :, None] * left[:, None]), 0.0) * inner
    sf = (k.reshape(n, h, nc * c, dk) * wf[..., None]).transpose(-1, -2) @ v.reshape(n, h, nc * c, dv)
    if init is not None:
        sf = sf + torch.exp(ld[None, :] * length)[:, :, None, None] * init
    return out, sf


def _plain_forward(s):
    o, sf = _decayed(s["q"], s["k"], s["v"], s["log_decay"], s["offsets"], s["max_len"], s["s0"], s["scale"], final=s["final"])
    return o.to(s["q"].dtype), sf


def _plain_backward(s):
    q, k, v, do, s0, ds = s["q"], s["k"], s["v"], s["do"], s["s0"], s["ds"]
    rest = (s["log_decay"], s["offsets"], s["max_len"])
    dq, _ = _decayed(do, v, k, *rest, None if s0 is None else s0.transpose(-1, -2), s["scale"])
    dv, ds0 = _decayed(k, q, do, *rest, ds, 1.0, reverse=True, inner=s["scale"], final=s0 is not None)
    dk, _ = _decayed(v, do, q, *rest, None if ds is None else ds.transpose(-1, -2), 1.0, reverse=True, inner=s["scale"])
    return dq.to(q.dtype), dk.to(q.dtype), dv.to(q.dtype), ds0


def _plain_step(s):
    at = s["slots"].long()
    q, k, v = s["q"].float(), s["k"].float(), s["v"].float()
    new = s["pool"][at] * torch.exp(s["log_decay"])[None, :, None, None] + k[..., :, None] * v[..., None, :]
    s["pool"][at] = new
    return ((q[..., :, None] * new).sum(-2) * s["scale"]).to(s["q"].dtype)


def _plain_layout(s):
    ctx, new, table, free, b, most = s["ctx_lens"], s["new_lens"], s["table"], s["free"], s["block"], s["max_tokens"]
    n, width = table.shape
    dev = ctx.device
    zero = torch.zeros(1, dtype=torch.int32, device=dev)
    offsets = torch.cat([zero, torch.cumsum(new, 0, dtype=torch.int32)])
    have, want = (ctx + b - 1) // b, (ctx + new + b - 1) // b
    base = torch.cat([zero, torch.cumsum(want - have, 0, dtype=torch.int32)])
    col = torch.arange(width, device=dev, dtype=torch.int32)[None, :]
    fresh = (col >= have[:, None]) & (col < want[:, None])
    take = (base[:-1, None] + col - have[:, None]).clamp(0, free.numel() - 1)
    table.copy_(torch.where(fresh, free[take.long()], table))
    t = torch.arange(most, device=dev, dtype=torch.int32)
    r = torch.searchsorted(offsets[1:].contiguous(), t, right=True)
    inside = r < n
    r = r.clamp(max=n - 1)
    pos = ctx[r] + t - offsets[r]
    slot = table[r, torch.where(inside, pos // b, 0).long()].long() * b + pos % b
    counts = torch.stack([offsets[-1], base[-1]])
    return {"offsets": offsets, "slots": torch.where(inside, slot, -1), "positions": torch.where(inside, pos, 0),
            "requests": torch.where(inside, r, -1).int(), "counts": counts, "table": table}


def _plain_verify(s):
    p, q, d, k = s["p"], s["q"], s["drafts"].long(), s["drafts"].shape[1]
    n, v, dev = p.shape[0], p.shape[2], p.device
    pd = p[:, :k].gather(2, d[..., None])[..., 0].float()
    qd = q.gather(2, d[..., None])[..., 0].float() if q is not None else torch.ones_like(pd)
    j = torch.arange(k, device=dev)[None, :]
    counts = s["counts"].long()[:, None]
    ok = (s["uniform"] * qd < pd) & (j < counts)
    taken = torch.cumprod(ok.int(), 1).sum(1)
    r = torch.arange(n, device=dev)
    row = p[r, taken].float()
    at = taken.clamp(max=k - 1)
    refused = (taken < counts[:, 0])[:, None]
    if q is not None:
        draft_row = q[r, at].float()
    else:
        draft_row = (torch.arange(v, device=dev)[None, :] == d[r, at][:, None]).float()
    left = torch.where(refused, (row - draft_row).clamp(min=0), row)
    score = left / s["noise"]
    # where rounding leaves nothing over, the target's own row decides
    score = torch.where((left > 0).any(1, keepdim=True), score, row / s["noise"])
    best = torch.where(score == score.amax(1, keepdim=True), torch.arange(v, device=dev)[None, :], v).amin(1)
    jj = torch.arange(k + 1, device=dev)[None, :]
    padded = torch.cat([d, torch.zeros_like(d[:, :1])], 1)
    tokens = torch.where(jj < taken[:, None], padded, torch.where(jj == taken[:, None], best[:, None], -1))
    return {"tokens": tokens.int(), "accepted": taken.int()}


# ----------------------------------------------------------------------------------------------------------------- run


def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_plain(s):
    op = s["op"]
    if op == "prompt":
        o, sf = _plain_forward(s)
        return {"o": o, "state": sf}
    if op == "train":
        o, sf = _plain_forward(s)
        dq, dk, dv, ds0 = _plain_backward(s)
        return {"o": o, "state": sf, "dq": dq, "dk": dk, "dv": dv, "dstate": ds0}
    if op == "step":
        return {"o": _plain_step(s), "pool": s["pool"]}
    return _plain_layout(s) if op == "layout" else _plain_verify(s)


def _run_own(s):
    import mapreduce_prefix_scan_gb300 as ak

    op = s["op"]
    if op in ("prompt", "train"):
        same = dict(offsets=s["offsets"], state=s["s0"], scale=s["scale"], max_len=s["max_len"])
        o, sf = ak.ak_linear_attention(s["q"], s["k"], s["v"], s["log_decay"], final_state=s["final"], **same)
        if op == "prompt":
            return {"o": o, "state": sf}
        dq, dk, dv, ds0 = ak.ak_linear_attention_backward(s["do"], s["q"], s["k"], s["v"], s["log_decay"], dstate_out=s["ds"], **same)
        return {"o": o, "state": sf, "dq": dq, "dk": dk, "dv": dv, "dstate": ds0}
    if op == "step":
        o = ak.ak_linear_attention_step(s["q"], s["k"], s["v"], s["log_decay"], s["pool"], slots=s["slots"], scale=s["scale"])
        return {"o": o, "pool": s["pool"]}
    if op == "layout":
        r = ak.ak_batch_layout(s["ctx_lens"], s["new_lens"], s["table"], s["free"], block_size=s["block"], max_tokens=s["max_tokens"])
        return {"offsets": r.offsets, "slots": r.slots, "positions": r.positions, "requests": r.requests, "counts": r.counts, "table": s["table"]}
    tokens, accepted = ak.ak_verify_drafts(s["p"], s["drafts"], s["uniform"], s["noise"], draft_probs=s["q"], draft_counts=s["counts"])
    return {"tokens": tokens, "accepted": accepted}


# --------------------------------------------------------------------------------------------------------------- exact


def exact(case, seed):
    s = prepare(case, seed)
    with torch.no_grad():
        if case["op"] in ("prompt", "train"):
            return _exact_attention(s, case["op"] == "train")
        if case["op"] == "step":
            return _exact_step(s)
        return _exact_layout(s) if case["op"] == "layout" else _exact_verify(s)


def _exact_attention(s, train):
    """Token by token from the recurrences, all sequences side by side."""
    lens, ld, scale = s["lens"], s["log_decay"].double(), s["scale"]
    n, (t, h, d), dev = len(lens), s["q"].shape, s["q"].device
    starts = np.concatenate([[0], np.cumsum(lens)[:-1]])
    order = np.argsort(-lens, kind="stable")  # longest first: the live sequences of a step are a prefix
    q, k, v = (s[x].double() for x in "qkv")
    w = torch.exp(ld)[None, :, None, None]
    S = torch.zeros(n, h, d, d, dtype=torch.float64, device=dev) if s["s0"] is None else s["s0"].double()[torch.as_tensor(order, device=dev)]
    S = S.clone()
    starts_t = torch.as_tensor(starts[order], device=dev)
    lens_t = torch.as_tensor(lens[order], device=dev)
    live = [int((lens > i).sum()) for i in range(int(lens.max()))]
    back = torch.as_tensor(np.argsort(order), device=dev)
    o = torch.zeros(t, h, d, dtype=torch.float64, device=dev)
    out = {}
    if train:
        do = s["do"].double()
        dq, dk, dv = torch.zeros_like(o), torch.zeros_like(o), torch.zeros_like(o)
    for i, m in enumerate(live):
        at = starts_t[:m] + i
        S[:m] = S[:m] * w + k[at][..., :, None] * v[at][..., None, :]
        o[at] = scale * (q[at][..., None, :] @ S[:m])[..., 0, :]
        if train:
            dq[at] = scale * (S[:m] @ do[at][..., :, None])[..., 0]
    out["o"] = o
    out["state"] = S[back] if s["final"] else None
    if train:
        G = torch.zeros_like(S) if s["ds"] is None else s["ds"].double()[torch.as_tensor(order, device=dev)].clone()
        for i, m in enumerate(live):
            at = starts_t[:m] + lens_t[:m] - 1 - i
            G[:m] += scale * q[at][..., :, None] * do[at][..., None, :]
            dv[at] = (k[at][..., None, :] @ G[:m])[..., 0, :]
            dk[at] = (G[:m] @ v[at][..., :, None])[..., 0]
            G[:m] *= w
        out |= {"dq": dq, "dk": dk, "dv": dv, "dstate": G[back] if s["s0"] is not None else None}
    return out


def _exact_step(s):
    pool, w = s["pool"].double(), torch.exp(s["log_decay"].double())
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device=pool.device)
    for b, slot in enumerate(s["slots"].tolist()):
        pool[slot] = w[:, None, None] * pool[slot] + torch.einsum("hi,hj->hij", s["k"][b].double(), s["v"][b].double())
        o[b] = s["scale"] * torch.einsum("hi,hij->hj", s["q"][b].double(), pool[slot])
    return {"o": o, "pool": pool}


def _exact_layout(s):
    ctx, new, table, free = (s[x].cpu().numpy().astype(np.int64) for x in ("ctx_lens", "new_lens", "table", "free"))
    b, most = s["block"], s["max_tokens"]
    slots, positions, requests = np.full(most, -1, np.int64), np.zeros(most, np.int32), np.full(most, -1, np.int32)
    offsets, at, taken = [0], 0, 0
    for r in range(len(ctx)):
        for c in range(-(-int(ctx[r]) // b), -(-int(ctx[r] + new[r]) // b)):
            table[r, c] = free[taken]
            taken += 1
        pos = ctx[r] + np.arange(new[r])
        to = slice(at, at + int(new[r]))
        positions[to], requests[to], slots[to] = pos, r, table[r, pos // b] * b + pos % b
        at += int(new[r])
        offsets.append(at)
    return {"offsets": np.array(offsets, np.int32), "slots": slots, "positions": positions, "requests": requests,
            "counts": np.array([at, taken], np.int32), "table": table.astype(np.int32)}


def _exact_verify(s):
    p, q, noise = s["p"], s["q"], s["noise"]
    drafts, counts, u = s["drafts"].tolist(), s["counts"].tolist(), s["uniform"].double().cpu().numpy()
    n, k = s["drafts"].shape
    tokens, accepted = np.full((n, k + 1), -1, np.int32), np.zeros(n, np.int32)
    at = s["drafts"].long()[..., None]
    pd = p[:, :k].gather(2, at)[..., 0].double().cpu().numpy()
    qd = np.ones((n, k)) if q is None else q.gather(2, at)[..., 0].double().cpu().numpy()
    for r in range(n):
        j = 0
        while j < counts[r] and u[r, j] * qd[r, j] < pd[r, j]:
            tokens[r, j] = drafts[r][j]
            j += 1
        left = p[r, j].double()
        if j < counts[r]:
            if q is None:
                left[drafts[r][j]] = 0.0
            else:
                left = (left - q[r, j].double()).clamp(min=0)
        if not bool((left > 0).any()):
            left = p[r, j].double()
        tokens[r, j] = int((left / noise[r].double()).argmax())
        accepted[r] = j
    return {"tokens": tokens, "accepted": accepted}
