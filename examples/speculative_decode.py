"""Speculative decoding of a batch of requests over one linear-attention layer, all sequence operators together.

Each round, for every request:

1. a drafter proposes ``k`` tokens, one at a time (``ak_linear_attention_step``
   on a copy of the states);
2. the target runs the last kept token and the drafts in one packed call
   (``ak_batch_layout`` for the offsets, ``ak_linear_attention`` from the states,
   which stay as they were);
3. ``ak_verify_drafts`` decides how many drafts are kept and which token follows;
4. the tokens that were kept enter the states in one ragged call, in place,
   and a paged log (``ak_batch_layout`` again: offsets, block tables and slots of
   the new lengths, computed on the device).

The weights are random. At the end the states are recomputed from each request's whole history, read back
through its block table.

    python examples/speculative_decode.py [--requests 24] [--rounds 12] [--drafts 4]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import mapreduce_prefix_scan_gb300 as ak  # noqa: E402


def run(requests=24, rounds=12, drafts=4, vocab=500, heads=4, dim=64, block=16, dtype=torch.bfloat16, seed=0):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)

    def normal(*shape, scale=1.0):
        return torch.randn(*shape, generator=g, device=dev) * scale

    n, k, width = requests, drafts, heads * dim
    embed = normal(vocab, 3, heads, dim).to(dtype)        # a token's q, k and v
    head = normal(width, vocab, scale=width**-0.5)         # the target's output layer
    head_q = head + normal(width, vocab, scale=0.3 * width**-0.5)  # the drafter's
    log_decay = -torch.exp2(-torch.arange(1, heads + 1, device=dev, dtype=torch.float32))
    scale = dim**-0.5

    def probs(o, w):
        return (o.float().reshape(o.shape[0], width) @ w).softmax(-1)

    state = torch.zeros(n, heads, dim, dim, device=dev)
    last = torch.randint(0, vocab, (n,), generator=g, device=dev, dtype=torch.int32)
    first = last.clone()
    ctx = torch.zeros(n, dtype=torch.int32, device=dev)    # tokens in the states and in the log
    pages = -(-rounds * (k + 1) // block)
    table = torch.full((n, pages), -1, dtype=torch.int32, device=dev)
    free = torch.randperm(n * pages, generator=g, device=dev).int()
    log = torch.full((n * pages * block,), -1, dtype=torch.int32, device=dev)
    all_new = torch.full((n,), k + 1, dtype=torch.int32, device=dev)
    scratch_table = torch.zeros(n, 1, dtype=torch.int32, device=dev)
    kept = 0

    for _ in range(rounds):
        # 1 the drafter
        s, token = state.clone(), last
        proposed, q_rows = [], []
        for _ in range(k):
            x = embed[token.long()]
            o = ak.ak_linear_attention_step(x[:, 0], x[:, 1], x[:, 2], log_decay, s, scale=scale)
            q_rows.append(probs(o, head_q))
            token = (q_rows[-1] / torch.empty_like(q_rows[-1]).exponential_(generator=g)).argmax(-1).int()
            proposed.append(token)
        proposed, q_rows = torch.stack(proposed, 1), torch.stack(q_rows, 1)

        # 2 the target over the last kept token and the drafts
        run_of = torch.cat([last[:, None], proposed], 1)
        layout = ak.ak_batch_layout(ctx, all_new, scratch_table, free[:0], block_size=block, max_tokens=n * (k + 1))
        x = embed[run_of.reshape(-1).long()]
        o, _ = ak.ak_linear_attention(x[:, 0], x[:, 1], x[:, 2], log_decay, offsets=layout.offsets, state=state,
                                      scale=scale, max_len=k + 1)
        p_rows = probs(o, head).reshape(n, k + 1, vocab)

        # 3 the decision
        noise = torch.empty(n, vocab, device=dev).exponential_(generator=g).clamp_(min=1e-20)
        tokens, accepted = ak.ak_verify_drafts(p_rows, proposed, torch.rand(n, k, generator=g, device=dev), noise,
                                               draft_probs=q_rows)

        # 4 what was kept enters the states and the log
        new = accepted + 1
        layout = ak.ak_batch_layout(ctx, new, table, free, block_size=block, max_tokens=n * (k + 1))
        used = layout.requests >= 0
        r = layout.requests.clamp(min=0).long()
        of_run = run_of[r, (layout.positions - ctx[r]).clamp(min=0).long()]
        x = embed[of_run.long()]
        ak.ak_linear_attention(x[:, 0], x[:, 1], x[:, 2], log_decay, offsets=layout.offsets, state=state, scale=scale,
                               state_out=state, max_len=k + 1)
        log[layout.slots[used]] = of_run[used]
        ctx = ctx + new
        free = free[int(layout.counts[1]):]
        last = tokens.gather(1, accepted.long()[:, None])[:, 0]
        kept += int(accepted.sum())

    # the whole history again, through the block tables
    lengths = ctx.tolist()
    history = []
    for i, m in enumerate(lengths):
        pos = torch.arange(m, device=dev)
        history.append(log[table[i, pos // block].long() * block + pos % block])
    offsets = torch.tensor([0] + lengths, device=dev).cumsum(0).int()
    x = embed[torch.cat(history).long()]
    _, again = ak.ak_linear_attention(x[:, 0], x[:, 1], x[:, 2], log_decay, offsets=offsets, scale=scale, final_state=True)
    return dict(lengths=lengths, kept=kept, proposed=n * k * rounds, state=state, again=again, first=first,
                history=history, free=free, table=table)


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--requests", type=int, default=24)
    ap.add_argument("--rounds", type=int, default=12)
    ap.add_argument("--drafts", type=int, default=4)
    a = ap.parse_args()
    r = run(a.requests, a.rounds, a.drafts)
    off = float((r["state"] - r["again"]).norm() / r["again"].norm())
    print(f"{a.requests} requests, {a.rounds} rounds: {r['kept']} of {r['proposed']} drafts kept, "
          f"{sum(r['lengths'])} tokens; states against a recomputation: {off:.1e} relative")


if __name__ == "__main__":
    main()
