"""Sliding-window attention with first tokens that stay visible, float64
(test infrastructure only; see the package docstring).

The query at position ``P`` sees position ``j`` when ``j <= P`` and
(``j < sinks`` or ``j > P - window``).  Every key of an extend, the suffix's
too, is read from the pool through ``req_to_token``.
"""
from __future__ import annotations

import numpy as np

from .attention import _kv_head_of, bf16_bits_to_f64, default_scale
from .fp8 import e4m3_decode


def visible_positions(P: int, window: int, sinks: int) -> np.ndarray:
    """Positions the query at position ``P`` sees, ascending."""
    j = np.arange(P + 1)
    return j[(j < sinks) | (j > P - window)]


def pool_reader(pool, scale=None):
    """slots -> float64 rows of a bf16 pool (bit patterns), or of an e4m3 pool
    when a scale is given."""
    if scale is None:
        return lambda slots: bf16_bits_to_f64(pool[slots])
    return lambda slots: e4m3_decode(pool[slots]) * float(scale)


def attend(q, read_k, read_v, row, P, window, sinks, num_kv_heads, scale, max_seq=None):
    """One query token (q [Hq, D] float64) at position ``P`` of the request
    whose slots are ``row``, over what it sees (below ``max_seq`` where that
    is given; 0 where that is nothing).  Returns (out [Hq, D], terms): ``terms`` holds,
    for each head, the sums an error bound is made of -- ``spread`` =
    sum_j p_j |V_j| [D], ``reach`` = max_j scale sum_d |q_d K_jd|, ``floor`` =
    keys * max|V| / sum_j exp(s_j - max s)."""
    pos = visible_positions(P, window, sinks)
    if max_seq is not None:
        pos = pos[pos < max_seq]
    slots = np.asarray(row, dtype=np.int64)[pos]
    K, V = read_k(slots), read_v(slots)
    Hq, D = q.shape
    out, spread = np.zeros((Hq, D)), np.zeros((Hq, D))
    reach, floor = np.zeros((Hq, 1)), np.zeros((Hq, 1))
    for h in range(Hq if pos.size else 0):
        kh = _kv_head_of(h, Hq, num_kv_heads)
        s = scale * (K[:, kh] @ q[h])
        w = np.exp(s - s.max())
        out[h] = (w @ V[:, kh]) / w.sum()
        spread[h] = (w @ np.abs(V[:, kh])) / w.sum()
        reach[h] = scale * (np.abs(K[:, kh]) @ np.abs(q[h])).max()
        floor[h] = pos.size * np.abs(V[:, kh]).max() / w.sum()
    return out, dict(spread=spread, reach=reach, floor=floor)


def _run(q, read_k, read_v, req_to_token, items, num_kv_heads, window, sinks, sm_scale, max_seq=None):
    q = np.asarray(q)
    scale = default_scale(q.shape[2]) if sm_scale is None else float(sm_scale)
    out = np.zeros(q.shape)
    terms = dict(spread=np.zeros(q.shape), reach=np.zeros(q.shape[:2] + (1,)), floor=np.zeros(q.shape[:2] + (1,)))
    for i, row, P in items:
        out[i], t = attend(bf16_bits_to_f64(q[i]), read_k, read_v, req_to_token[int(row)], int(P), int(window),
                           int(sinks), num_kv_heads, scale, max_seq)
        for k in terms:
            terms[k][i] = t[k]
    return out, terms


def decode_attention_window(q, read_k, read_v, req_to_token, req_pool_idx, seq_lens, num_kv_heads, window, sinks,
                            sm_scale=None, max_seq=None):
    """(out [B, Hq, D], error terms); rows of requests without keys are 0.
    ``max_seq``: positions from it on are left out of what a query sees."""
    items = [(r, req_pool_idx[r], int(n) - 1) for r, n in enumerate(seq_lens) if n > 0]
    return _run(q, read_k, read_v, req_to_token, items, num_kv_heads, window, sinks, sm_scale, max_seq)


def extend_attention_window(q, read_k, read_v, req_to_token, req_pool_idx, prefix_lens, extend_lens, num_kv_heads,
                            window, sinks, sm_scale=None, tokens=None):
    """(out [T, Hq, D], error terms); ``tokens``: the rows computed (others 0)."""
    items, at = [], 0
    for r, (p, e) in enumerate(zip(prefix_lens, extend_lens)):
        items += [(at + i, req_pool_idx[r], int(p) + i) for i in range(int(e))]
        at += int(e)
    if tokens is not None:
        keep = set(int(t) for t in tokens)
        items = [x for x in items if x[0] in keep]
    return _run(q, read_k, read_v, req_to_token, items, num_kv_heads, window, sinks, sm_scale)
