"""Plain 64-bit implementations of the sequence operators (numpy), written
from their definitions, and the error bounds their tests use."""
from __future__ import annotations

import numpy as np


def layout(ctx, new, table, free, block, max_tokens):
    """Block tables, slot map and packed offsets, request by request."""
    ctx = [max(int(x), 0) for x in ctx]
    new = [max(int(x), 0) for x in new]
    table = np.array(table, dtype=np.int64)
    width = table.shape[1]
    slots = np.full(max_tokens, -1, np.int64)
    positions = np.zeros(max_tokens, np.int64)
    requests = np.full(max_tokens, -1, np.int64)
    offsets, at, taken = [0], 0, 0
    for r in range(len(ctx)):
        for c in range(-(-ctx[r] // block), -(-(ctx[r] + new[r]) // block)):
            if c < width:
                table[r, c] = free[taken] if taken < len(free) else -1
            taken += 1
        for i in range(new[r]):
            if at + i < max_tokens:
                pos = ctx[r] + i
                positions[at + i], requests[at + i] = pos, r
                col = pos // block
                if col < width and table[r, col] >= 0:
                    slots[at + i] = table[r, col] * block + pos % block
        at += new[r]
        offsets.append(at)
    return np.array(offsets), slots, positions, requests, np.array([at, taken]), table


def verify(p, q, drafts, counts, u, noise):
    """Kept drafts and the token after them; p, q, noise as stored (float32 values)."""
    n, k = drafts.shape
    vocab = p.shape[2]
    tokens, accepted = np.full((n, k + 1), -1, np.int64), np.zeros(n, np.int64)
    for r in range(n):
        m = k if counts is None else min(max(int(counts[r]), 0), k)
        j = 0
        while j < m:
            d = drafts[r, j]
            if not 0 <= d < vocab:
                break
            qd = np.float32(1) if q is None else q[r, j, d]
            if not float(u[r, j]) * float(qd) < float(p[r, j, d]):
                break
            tokens[r, j] = d
            j += 1
        left = p[r, j].astype(np.float64)
        if j < m:
            if q is not None:
                left = left - q[r, j].astype(np.float64)
            elif 0 <= drafts[r, j] < vocab:
                left[drafts[r, j]] = 0
        for w in (left, p[r, j].astype(np.float64)):
            with np.errstate(all="ignore"):
                score = np.where(w > 0, w / noise[r].astype(np.float64), np.nan)
            score = np.where(score >= 0, score, -1)  # NaN and negative scores are no candidates
            if (score >= 0).any():
                tokens[r, j] = int(np.argmax(score))
                break
        accepted[r] = j
    return tokens, accepted


def attention(q, k, v, ld, offsets, s0=None, scale=1.0):
    """o, final states and, per output, the sum of absolute values of what its last two products add up."""
    t, h, _ = q.shape
    dv = v.shape[2]
    n = len(offsets) - 1
    g = np.exp(ld.astype(np.float64))
    o, mass = np.zeros((t, h, dv)), np.zeros((t, h, dv))
    sf = np.zeros((n, h, q.shape[2], dv))
    for s in range(n):
        for x in range(h):
            S = np.zeros((q.shape[2], dv)) if s0 is None else s0[s, x].astype(np.float64)
            A = np.abs(S)
            for i in range(offsets[s], offsets[s + 1]):
                S = g[x] * S + np.outer(k[i, x], v[i, x])
                A = g[x] * A + np.outer(np.abs(k[i, x]), np.abs(v[i, x]))
                o[i, x] = scale * (q[i, x] @ S)
                mass[i, x] = abs(scale) * (np.abs(q[i, x]) @ A)
            sf[s, x] = S
    return o, sf, mass


def attention_gradients(do, q, k, v, ld, offsets, s0=None, ds=None, scale=1.0):
    """dq, dk, dv, dS_0 of sum(o * do) + sum(S_T * ds), from the recurrences."""
    t, h, dk_ = q.shape
    dv_ = v.shape[2]
    n = len(offsets) - 1
    g = np.exp(ld.astype(np.float64))
    dq, dk, dv = np.zeros(q.shape), np.zeros(k.shape), np.zeros(v.shape)
    d0 = np.zeros((n, h, dk_, dv_))
    for s in range(n):
        for x in range(h):
            S = np.zeros((dk_, dv_)) if s0 is None else s0[s, x].astype(np.float64)
            for i in range(offsets[s], offsets[s + 1]):
                S = g[x] * S + np.outer(k[i, x], v[i, x])
                dq[i, x] = scale * (S @ do[i, x])
            G = np.zeros((dk_, dv_)) if ds is None else ds[s, x].astype(np.float64)
            for i in range(offsets[s + 1] - 1, offsets[s] - 1, -1):
                G = G + scale * np.outer(q[i, x], do[i, x])
                dk[i, x] = G @ v[i, x]
                dv[i, x] = k[i, x] @ G
                G = g[x] * G
            d0[s, x] = G
    return dq, dk, dv, d0
