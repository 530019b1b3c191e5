"""Seeded inputs of the drafted-token tests, and the error bounds they allow."""
from __future__ import annotations

import numpy as np

import oracle
from radixattention_prefix_shared_gb300 import workloads as W


def tree(g, n, kind):
    """Parents of a request's nodes: a chain, a bush (all below the root), a random
    tree, or a forest (some nodes without a parent)."""
    if n == 0:
        return []
    if kind == "chain":
        return [i - 1 for i in range(n)]
    if kind == "bush":
        return [-1] + [0] * (n - 1)
    if kind == "forest":
        return [int(g.integers(-1, i)) if i else -1 for i in range(n)]
    return [-1] + [int(g.integers(max(0, i - 4), i)) for i in range(1, n)]


def attention_case(seed, *, Hq, Hkv, D, prefix, drafts, kind="tree", shared=0, fp8=False, std=1.0, spare=17):
    """A batch of ``drafts[r]`` nodes after ``prefix[r]`` tokens; the first ``shared``
    slots are the same in every row with nodes.  Pool rows that no position of the
    batch holds are NaN, and all other entries of req_to_token point at those."""
    g = np.random.default_rng(seed)
    n = [max(0, x) for x in drafts]
    live = shared + sum(p - shared + x for p, x in zip(prefix, n) if x)
    S = live + spare
    perm = g.permutation(S).astype(np.int32)
    slots, dead = perm[:live], perm[live:]
    rows, stride = len(n) + 3, max(p + x for p, x in zip(prefix, n)) + 2
    rtt = dead[g.integers(0, dead.size, size=(rows, stride))].astype(np.int32)
    rpi = g.permutation(rows)[: len(n)].astype(np.int32)
    at = shared
    for r, (p, x) in enumerate(zip(prefix, n)):
        if x:
            rtt[rpi[r], :shared] = slots[:shared]
            rtt[rpi[r], shared: p + x] = slots[at: at + p + x - shared]
            at += p + x - shared
        else:   # a padding row names no row of the table
            rpi[r] = -7
    par = [v for x in n for v in tree(g, x, kind)]
    c = dict(Hq=Hq, Hkv=Hkv, D=D, S=S, shared=shared, rtt=rtt, rpi=rpi, prefix=np.asarray(prefix, np.int32),
             drafts=np.asarray(drafts, np.int32), parents=np.asarray(par or [-1], np.int32), fp8=fp8, k_scale=None,
             v_scale=None)
    c["q"] = W.f32_to_bf16_bits((g.standard_normal((max(1, sum(n)), Hq, D)) * std).astype(np.float32))
    k, v = (W.f32_to_bf16_bits((g.standard_normal((S, Hkv, D)) * std).astype(np.float32)) for _ in range(2))
    if fp8:
        c["k_scale"], c["v_scale"] = 1 / 32 * std, 0.0173
        k, v = oracle.fp8.quantize(k, c["k_scale"]), oracle.fp8.quantize(v, c["v_scale"])
    k[dead], v[dead] = (0x7F, 0x7F) if fp8 else (0x7FFF, 0x7FFF)
    c["pool_k"], c["pool_v"] = k, v
    return c


def want_attention(c):
    return oracle.drafts.verify_attention(
        c["q"], oracle.window.pool_reader(c["pool_k"], c["k_scale"]), oracle.window.pool_reader(c["pool_v"], c["v_scale"]),
        c["rtt"], c["rpi"], c["prefix"], c["drafts"], c["parents"], c["Hkv"])


def assert_attention(got_bits, c, what=""):
    """Largest error a correct kernel makes, value by value.

    The output is rounded to bf16 (2^-8 of it).  The weights go to the tensor core
    in bf16 (2^-8 of each; f16 over e4m3 pools, less), which moves the sum by 2^-8 of
    ``spread`` = sum p |V|.  Scores: fp32 dots of at most 128 terms are off by 2^-17 of
    ``reach`` = sum |q k| scale; a score off by d moves every weight by d and the output
    by 2 d of ``spread``.  The approximate exponentials, the fp32 sums and the merges
    add less than 2^-12 of ``spread`` together.  f16 weights below 2^-32 of the largest
    of their segment round to nothing: at most 2^-32 of ``floor`` = keys max|V| / sum p."""
    got = oracle.bf16_bits_to_f64(got_bits)
    want, terms = want_attention(c)
    rows = int(np.maximum(c["drafts"], 0).sum())
    got, want = got[:rows], want[:rows]
    bound = (2.0 ** -8 * np.abs(want) + (2.0 ** -8 + 2.0 ** -12 + 2.0 ** -16 * terms["reach"][:rows])
             * terms["spread"][:rows] + 2.0 ** -32 * terms["floor"][:rows] + 1e-30)
    assert np.isfinite(got).all(), f"{what}: non-finite output (a hidden position was read?)"
    ratio = np.abs(got - want) / bound
    assert ratio.size == 0 or ratio.max() <= 1.0, \
        f"{what}: error {ratio.max():.3g} of its bound at {np.unravel_index(ratio.argmax(), ratio.shape)}"


def softmax_rows(g, n, V, std=3.0, base=None):
    x = g.standard_normal((n, V)) * std if base is None else base + g.standard_normal((n, V))
    e = np.exp(x - x.max(-1, keepdims=True))
    return (e / e.sum(-1, keepdims=True)).astype(np.float32), x


def accept_case(seed, *, drafts, V, kind="tree", drawn=True):
    """Trees whose tokens were drawn from the draft rows of their parents, or picked."""
    g = np.random.default_rng(seed)
    n = [max(0, x) for x in drafts]
    T = max(1, sum(n))
    p, base = softmax_rows(g, T, V)
    q, _ = softmax_rows(g, T, V, base=base)
    par = [v for x in n for v in tree(g, x, kind)] or [-1]
    starts = np.repeat(np.cumsum([0] + n)[:-1], n)
    tok = np.zeros(T, np.int32)
    for t, s in enumerate(starts):
        row = q[s + max(0, par[t])].astype(np.float64)
        tok[t] = g.choice(V, p=row / row.sum()) if drawn else np.argsort(-row)[g.integers(0, min(V, 4))]
    return dict(V=V, p=p, q=q if drawn else None, tok=tok, parents=np.asarray(par, np.int32),
                drafts=np.asarray(drafts, np.int32), coins=g.random(T).astype(np.float32),
                final=g.random(len(drafts)).astype(np.float32), most=max(1, max(n, default=1)))


def want_accept(c):
    return oracle.drafts.verify_drafts(c["p"], c["q"], c["tok"], c["parents"], c["drafts"], c["coins"], c["final"],
                                       c["most"])
