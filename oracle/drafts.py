"""A step over drafted tokens, float64 (test infrastructure only; see the package
docstring): attention of a request's tree of drafted tokens, the walk down the
tree against the target's probabilities, and what becomes of the tokens' slots.

A request's nodes are consecutive tokens; ``parents`` holds each node's parent
among them, and any value outside [0, node) stands for none.
"""
from __future__ import annotations

import numpy as np

from .attention import _kv_head_of, bf16_bits_to_f64, default_scale


def line_of(parents, i):
    """Node ``i`` and the nodes above it, ascending."""
    line = [i]
    while 0 <= parents[line[-1]] < line[-1]:
        line.append(int(parents[line[-1]]))
    return line[::-1]


def verify_attention(q, read_k, read_v, req_to_token, req_pool_idx, prefix_lens, draft_lens, parents, num_kv_heads,
                     sm_scale=None):
    """(out [T, Hq, D], error terms as ``oracle.window.attend`` gives them)."""
    q = np.asarray(q)
    T, Hq, D = q.shape
    scale = default_scale(D) if sm_scale is None else float(sm_scale)
    out = np.zeros(q.shape)
    terms = dict(spread=np.zeros(q.shape), reach=np.zeros((T, Hq, 1)), floor=np.zeros((T, Hq, 1)))
    off = 0
    for r, n in enumerate(draft_lens):
        n = max(0, int(n))
        if n == 0:
            continue
        p, par = int(prefix_lens[r]), parents[off: off + n]
        slots = np.asarray(req_to_token[int(req_pool_idx[r])][: p + n], dtype=np.int64)
        K, V = read_k(slots), read_v(slots)
        for i in range(n):
            pos = np.concatenate([np.arange(p), p + np.asarray(line_of(par, i))])
            qi = bf16_bits_to_f64(q[off + i])
            for h in range(Hq):
                kh = _kv_head_of(h, Hq, num_kv_heads)
                k, v = K[pos, kh], V[pos, kh]
                s = scale * (k @ qi[h])
                w = np.exp(s - s.max())
                out[off + i, h] = (w @ v) / w.sum()
                terms["spread"][off + i, h] = (w @ np.abs(v)) / w.sum()
                terms["reach"][off + i, h] = scale * (np.abs(k) @ np.abs(qi[h])).max()
                terms["floor"][off + i, h] = pos.size * np.abs(v).max() / w.sum()
        off += n
    return out, terms


def _weights(row):
    row = np.asarray(row, dtype=np.float64)
    return np.where(np.isfinite(row) & (row > 0), row, 0.0)


def walk(target, draft, tokens, parents, coins, final_coin):
    """One request: (kept nodes, next token).  ``target`` and ``draft`` (None:
    drafts were picked) hold a row a node."""
    V = len(target[0])
    kept, c, R, m = [0], 0, _weights(target[0]), 1.0
    for i in range(1, len(tokens)):
        if parents[i] != c or not 0 <= parents[i] < i:
            continue
        x = int(tokens[i])
        there = 0 <= x < V
        w = R[x] if there else 0.0
        q = 1.0 if draft is None else (_weights(draft[c])[x] if there else 0.0)
        if w > 0 and float(coins[i]) * q * m < w:
            c, R, m = i, _weights(target[i]), 1.0
            kept.append(i)
        elif draft is None:
            R = R.copy()
            if there:
                R[x] = 0.0
            m -= w
        else:
            R = np.maximum((R / m if m > 0 else 0 * R) - _weights(draft[c]), 0.0)
            m = R.sum()
    if not R.sum() > 0:
        R = _weights(target[c])
    if not R.sum() > 0:
        return kept, -1
    cum = np.cumsum(R)
    past = np.nonzero(cum > float(final_coin) * cum[-1])[0]
    return kept, int(past[0]) if past.size else int(np.nonzero(R)[0][-1])


def verify_drafts(target, draft, tokens, parents, draft_lens, coins, final_coins, max_draft):
    """(accepted [B, max_draft], num_accepted [B], next_tokens [B])."""
    B = len(draft_lens)
    accepted = np.full((B, max_draft), -1, np.int32)
    count, nxt = np.zeros(B, np.int32), np.full(B, -1, np.int32)
    off = 0
    for r, n in enumerate(draft_lens):
        n = max(0, int(n))
        if n:
            at = slice(off, off + n)
            kept, nxt[r] = walk(target[at], None if draft is None else draft[at], tokens[at], parents[at], coins[at],
                                final_coins[r])
            accepted[r, : len(kept)] = kept
            count[r] = len(kept)
        off += n
    return accepted, count, nxt


def commit_drafts(req_to_token, req_pool_idx, prefix_lens, draft_lens, slots, accepted, num_accepted):
    """(req_to_token, seq_lens, freed slots), the table a copy."""
    table, freed, off = np.array(req_to_token), [], 0
    seq = np.array(prefix_lens, np.int32)
    for r, n in enumerate(draft_lens):
        n = max(0, int(n))
        kept = [int(x) for x in accepted[r][: int(num_accepted[r])]] if n else []
        for k, i in enumerate(kept):
            table[int(req_pool_idx[r]), int(prefix_lens[r]) + k] = slots[off + i]
        seq[r] += len(kept)
        freed += [int(slots[off + i]) for i in range(n) if i not in kept]
        off += n
    return table, seq, np.asarray(freed, np.int32)
