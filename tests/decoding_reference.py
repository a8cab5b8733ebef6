"""Plain 64-bit implementations of the gated recurrence, beam search and block operators (numpy), written from their
definitions."""
from __future__ import annotations

import numpy as np


def weights(gate, form):
    with np.errstate(over="ignore"):
        if form == "decay":
            return np.exp(gate), np.ones_like(gate)
        return 1 / (1 + np.exp(-gate)), 1 / (1 + np.exp(gate))


def recurrence(x, gate, offsets, s0=None, form="decay"):
    """h, the final states, and per value the sum of absolute values of what it adds up."""
    a, b = weights(gate, form)
    h, mass = np.zeros_like(x), np.zeros_like(x)
    n = len(offsets) - 1
    sf = np.zeros((n, x.shape[1]))
    for s in range(n):
        S = np.zeros(x.shape[1]) if s0 is None else s0[s].copy()
        A = np.abs(S)
        for t in range(offsets[s], offsets[s + 1]):
            S = a[t] * S + b[t] * x[t]
            A = a[t] * A + b[t] * np.abs(x[t])
            h[t], mass[t] = S, A
        sf[s] = S
    return h, sf, mass


def recurrence_gradients(dh, x, gate, offsets, s0=None, ds=None, form="decay"):
    """dx, dgate, dS_0 of sum(h dh) + sum(S_T ds), and the masses of G and of h_{t-1}."""
    a, b = weights(gate, form)
    h, _, hm = recurrence(x, gate, offsets, s0, form)
    n = len(offsets) - 1
    dx, dg, gm, before = np.zeros_like(x), np.zeros_like(x), np.zeros_like(x), np.zeros_like(x)
    d0 = np.zeros((n, x.shape[1]))
    for s in range(n):
        lo, hi = offsets[s], offsets[s + 1]
        G = np.zeros(x.shape[1]) if ds is None else ds[s].copy()
        M = np.abs(G)
        for t in range(hi - 1, lo - 1, -1):
            G, M = G + dh[t], M + np.abs(dh[t])
            if t > lo:
                hp, before[t] = h[t - 1], hm[t - 1]
            else:
                hp = np.zeros(x.shape[1]) if s0 is None else s0[s]
                before[t] = np.abs(hp)
            dx[t], gm[t] = b[t] * G, M
            dg[t] = G * a[t] * hp if form == "decay" else G * (hp - x[t]) * a[t] * b[t]
            G, M = a[t] * G, a[t] * M
        d0[s] = G
    return dx, dg, d0, gm, before


def beam_step(logits, scores, done=None, lengths=None, end=-1, penalty=0.0, keep=None):
    """The best `keep` continuations of each request: scores, tokens, parents, done, lengths."""
    n, k, v = logits.shape
    keep = k if keep is None else keep
    out = (np.full((n, keep), -np.inf), np.full((n, keep), -1), np.full((n, keep), -1), np.ones((n, keep), bool), np.zeros((n, keep), int))
    for r in range(n):
        found = []
        for j in range(k):
            s, length = float(scores[r, j]), 0 if lengths is None else int(lengths[r, j])
            was = done is not None and bool(done[r, j])
            if not np.isfinite(s):
                continue
            with np.errstate(all="ignore"):
                if was:
                    cands = [(s, max(end, 0))]
                else:
                    length += 1
                    x = logits[r, j].astype(np.float64)
                    top = x.max()
                    if not np.isfinite(top):
                        continue  # a NaN, an infinity, or nothing
                    lse = top + np.log(np.exp(x - top).sum())
                    best = np.lexsort((np.arange(v), -x))[:keep]
                    cands = [(s + (x[t] - lse), int(t)) for t in best if x[t] > -np.inf]
                for total, t in cands:
                    rank = np.float64(total) / np.float64(length) ** penalty if penalty else total
                    if np.isfinite(rank):
                        found.append((-rank, j, t, total, was, length))
        for q, (_, j, t, total, was, length) in enumerate(sorted(found)[:keep]):
            t = end if was else t
            out[0][r, q], out[1][r, q], out[2][r, q] = total, t, j
            out[3][r, q], out[4][r, q] = was or (end >= 0 and t == end), length
    return out


def held(length, block, width):
    return min(-(-max(int(length), 0) // block), width)


def count(table, lens, block, blocks):
    refs = np.zeros(blocks, np.int64)
    for row, m in zip(table, lens):
        for i in row[: held(m, block, len(row))]:
            if 0 <= i < blocks:
                refs[i] += 1
    return refs


def fork(table, lens, parents, free, block, blocks):
    """table, lens, refs, pairs, [copies wanted]."""
    n, width = len(parents), table.shape[1]
    new, new_lens = np.full((n, width), -1, np.int64), np.zeros(n, np.int64)
    for r, p in enumerate(parents):
        if 0 <= p < len(lens):
            new_lens[r] = max(int(lens[p]), 0)
            m = held(lens[p], block, width)
            new[r, :m] = table[p, :m]
    refs = count(new, new_lens, block, blocks)
    tails = {}
    for r in range(n):
        col = int(new_lens[r]) // block
        if new_lens[r] % block and col < width and 0 <= new[r, col] < blocks:
            tails.setdefault(int(new[r, col]), []).append(r)
    # (a block that one row holds twice counts twice, and its end once)
    copies = sorted(r for i, rows in tails.items() for r in (rows[1:] if refs[i] <= len(rows) else rows))
    pairs = np.full((n, 2), -1, np.int64)
    for at, r in enumerate(copies):
        col = int(new_lens[r]) // block
        src = int(new[r, col])
        to = int(free[at]) if at < len(free) and 0 <= free[at] < blocks else -1
        refs[src] -= 1
        new[r, col] = to
        if to >= 0:
            refs[to] += 1
            pairs[at] = src, to
    return new, new_lens, refs, pairs, np.array([len(copies)])


def free_list(refs):
    ids = np.flatnonzero(np.asarray(refs) <= 0)
    out = np.full(len(refs), -1, np.int64)
    out[: len(ids)] = ids
    return out, np.array([len(ids)])


def compact(table, lens, refs, block):
    """table, pairs, [moves, blocks in use]."""
    blocks = len(refs)
    used = [i for i in range(blocks) if refs[i] > 0]
    n = len(used)
    moves = list(zip([i for i in used if i >= n], [i for i in range(n) if refs[i] <= 0]))
    to = dict(moves)
    out = np.array(table, np.int64)
    for r, m in enumerate(lens):
        for c in range(held(m, block, out.shape[1])):
            out[r, c] = to.get(int(out[r, c]), int(out[r, c]))
    pairs = np.full((blocks // 2, 2), -1, np.int64)
    pairs[: len(moves)] = np.array(moves, np.int64).reshape(-1, 2)
    return out, pairs, np.array([len(moves), n])
