"""Seeded inputs of the sliding-window tests, and the error bounds they allow."""
from __future__ import annotations

import numpy as np

import oracle
from radixattention_prefix_shared_gb300 import workloads as W


def attention_case(seed, *, Hq, Hkv, D, prefix, ext, window, sinks, fp8=False, std=1.0, spare=17):
    """A batch of ``ext[r]`` queries after ``prefix[r]`` tokens (a decode:
    ext 1, prefix seq_len - 1; seq_len 0: prefix 0, ext 0 with one q row).

    Slots of visible positions are a seeded permutation; every other pool row
    is NaN (bf16 0x7FFF, e4m3 0x7F) and every other entry of req_to_token
    points at one of those rows."""
    g = np.random.default_rng(seed)
    seq = [p + e for p, e in zip(prefix, ext)]
    spans = []
    for p, e in zip(prefix, ext):
        seen = np.unique(np.concatenate([oracle.window.visible_positions(P, window, sinks)
                                         for P in sorted({p, max(p, p + e - 1)})] or [[]])) if e else np.zeros(0, int)
        if e > 1:   # the union over the queries between
            lo = max(0, p - window + 1)
            seen = np.concatenate([np.arange(min(sinks, lo)), np.arange(lo, p + e)])
        spans.append(seen.astype(np.int64))
    live = sum(len(s) for s in spans)
    S = live + spare
    perm = g.permutation(S).astype(np.int32)
    slots, dead = perm[:live], perm[live:]
    rows, stride = len(ext) + 3, max(seq + [1]) + 2
    rtt = dead[g.integers(0, dead.size, size=(rows, stride))].astype(np.int32)
    rpi = g.permutation(rows)[: len(ext)].astype(np.int32)
    at = 0
    for r, s in enumerate(spans):
        rtt[rpi[r], s] = slots[at: at + len(s)]
        at += len(s)
    c = dict(Hq=Hq, Hkv=Hkv, D=D, S=S, window=window, sinks=sinks, rtt=rtt, rpi=rpi, prefix=np.asarray(prefix, np.int32),
             ext=np.asarray(ext, np.int32), seq=np.asarray(seq, np.int32), fp8=fp8, k_scale=None, v_scale=None)
    c["q"] = W.f32_to_bf16_bits((g.standard_normal((max(1, sum(ext)), Hq, D)) * std).astype(np.float32))
    k, v = (W.f32_to_bf16_bits((g.standard_normal((S, Hkv, D)) * std).astype(np.float32)) for _ in range(2))
    if fp8:
        c["k_scale"], c["v_scale"] = 1 / 32 * std, 0.0173
        k, v = oracle.fp8.quantize(k, c["k_scale"]), oracle.fp8.quantize(v, c["v_scale"])
    k[dead], v[dead] = (0x7F, 0x7F) if fp8 else (0x7FFF, 0x7FFF)
    c["pool_k"], c["pool_v"] = k, v
    return c


def readers(c):
    return (oracle.window.pool_reader(c["pool_k"], c["k_scale"]), oracle.window.pool_reader(c["pool_v"], c["v_scale"]))


def attention_bound(want, terms, fp8):
    """Largest error a correct kernel makes, value by value.

    The output is rounded to bf16 (2^-8 of it).  The weights P go to the
    tensor core in bf16, or as two e4m3 terms (2^-8 of each, which moves the
    sum by 2^-8 of ``spread`` = sum p |V|).  Scores: fp32 dots of at most 128
    terms are off by 128 * 2^-24 = 2^-17 of ``reach`` = sum |q k| scale; an
    e4m3 pool's query goes to the tensor core as three e4m3 terms, 2^-12 of
    each value.  A score off by d moves every weight by d and the output by
    2 d of ``spread``.  The approximate exponentials, the fp32 sums and the
    split merges add less than 2^-12 of ``spread`` together.  e4m3 P terms
    below 2^-18 of the largest weight round to nothing: at most 2^-18 of
    ``floor`` = keys max|V| / sum p (bf16 and f16 P reach far lower)."""
    score = terms["reach"] * (2.0 ** -12 if fp8 else 2.0 ** -17)
    bound = 2.0 ** -8 * np.abs(want) + (2.0 ** -8 + 2.0 ** -12 + 2 * score) * terms["spread"]
    if fp8:
        bound = bound + 2.0 ** -18 * terms["floor"]
    return bound + 1e-30


def assert_within(got_bits, want, terms, fp8, rows=None, what=""):
    got = oracle.bf16_bits_to_f64(got_bits)
    bound = attention_bound(want, terms, fp8)
    if rows is not None:
        got, want, bound = got[rows], want[rows], bound[rows]
    assert np.isfinite(got).all(), f"{what}: non-finite output (a hidden position was read?)"
    ratio = np.abs(got - want) / bound
    worst = np.unravel_index(ratio.argmax(), ratio.shape)
    assert ratio.max() <= 1.0, f"{what}: error {ratio.max():.3g} of its bound at {worst}"
    return float(ratio.max())
