"""What each path of the sliding-window calls rounds, and no more.

_window.py's bound is one for all paths over an e4m3 pool.  Here every path is
held to its own.  With u the relative half step of the weights P in the
product P.V, f the half step of the smallest ones against a request's largest,
and t that of the query in q.K:

  path                                                    u      f      t
  decode, bf16 pool, 1 or 2 query heads a KV head         0      0      0
  decode, bf16 pool, 3 and more (P in bf16)               2^-8   0      0
  decode, e4m3 pool, 1 query head                         0      0      0
  decode, e4m3 pool, 2 or 4 (P in two e4m3 terms, the     2^-8   2^-23  2^-12
    second 32 times its size; the query in three)
  decode, e4m3 pool, other groups (P in f16)              2^-11  2^-25  0
  extend, bf16 pool (P in bf16)                           2^-8   0      0
  extend, e4m3 pool (P in f16)                            2^-11  2^-25  0

(Two terms: hi is off by 2^-4 of x at most, and lo by 2^-4 of that, or by half
of e4m3's smallest step of 2^-9, over 32, in units of 2^-8 of the largest
weight: 2^-10 / 32 / 2^8 = 2^-23.  The f16 paths' reference of the exponentials
is never above the largest weight, so their subnormals' 2^-25 is of it or less.
bf16 has no subnormals to speak of.  A query of an e4m3 pool is exact in f16
from 2^-14 on; the inputs here hold nothing below but zero.)

An output is then off by 2^-8 of itself (bf16), by u + 2^-12 + 2 (t + 2^-17)
reach of ``spread`` and by f of ``floor`` (see _window.attention_bound for the
terms)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import oracle  # noqa: E402
from radixattention_prefix_shared_gb300 import workloads as W  # noqa: E402

from _window import attention_case  # noqa: E402
from test_gpu_window import Case  # noqa: E402

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]


def virtual_group(Hq, Hkv):
    """Query heads that share a KV head in the decode kernels (at most 16)."""
    g = Hq // Hkv
    return next(g // s for s in range(1, g + 1) if g % s == 0 and g // s <= 16)


def rounding(kind, fp8, Hq, Hkv):
    """(u, f, t) of a path."""
    g = virtual_group(Hq, Hkv)
    if kind == "decode" and (g == 1 or (g == 2 and not fp8)):
        return 0.0, 0.0, 0.0
    if not fp8:
        return 2.0 ** -8, 0.0, 0.0
    if kind == "decode" and g in (2, 4):
        return 2.0 ** -8, 2.0 ** -23, 2.0 ** -12
    return 2.0 ** -11, 2.0 ** -25, 0.0


def check(kind, c, out, want, terms, what=""):
    u, f, t = rounding(kind, c["fp8"], c["Hq"], c["Hkv"])
    score = (t + 2.0 ** -17) * terms["reach"]
    bound = 2.0 ** -8 * np.abs(want) + (u + 2.0 ** -12 + 2 * score) * terms["spread"] + f * terms["floor"] + 1e-30
    ratio = np.abs(oracle.bf16_bits_to_f64(W.bf16_bits(out)) - want) / bound
    assert ratio.max() <= 1.0, f"{kind} {what}: {ratio.max():.3g} of its bound"


def no_tiny_queries(c):
    q = oracle.bf16_bits_to_f64(c["q"])
    c["q"][np.abs(q) < 2.0 ** -14] = 0
    return c


def run_both(c, what):
    case = Case(c)
    if (c["ext"] == 1).all():
        check("decode", c, case.decode(), *case.want_decode(), what)
    check("extend", c, case.extend(), *case.want_extend(), what)


HEADS = [(4, 4, 128), (4, 4, 64), (8, 4, 128), (8, 4, 64), (6, 2, 128), (8, 2, 64), (16, 4, 128), (10, 2, 64),
         (16, 2, 128), (32, 2, 64), (34, 2, 64), (36, 2, 128)]


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("heads", HEADS, ids=lambda h: f"{h[0]}q{h[1]}kv{h[2]}d")
def test_single_tokens(heads, fp8):
    """Narrow and wide scores, one run a request and several."""
    Hq, Hkv, D = heads
    for window, std in ((200, 1.0), (900, 1.0), (200, 4.0)):
        c = attention_case(Hq + D, Hq=Hq, Hkv=Hkv, D=D, prefix=[40, 3000, 250, 700], ext=[1] * 4, window=window,
                           sinks=4, fp8=fp8, std=std)
        run_both(no_tiny_queries(c), f"window {window} std {std}")


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
def test_chunks(fp8):
    for Hq, Hkv, D, prefix, ext in ((8, 4, 128, [900, 3], [70, 130]), (6, 2, 64, [0, 500], [40, 33]),
                                    (80, 40, 64, [300, 30, 7], [60, 9, 20])):
        c = attention_case(Hq, Hq=Hq, Hkv=Hkv, D=D, prefix=prefix, ext=ext, window=250, sinks=3, fp8=fp8)
        run_both(no_tiny_queries(c), f"{Hq} on {Hkv}")


def sink_case(seed, nats, *, Hq, Hkv, D, batch, window, sinks, fp8):
    """Single tokens whose first ``sinks`` keys score ``nats`` above the window's
    and whose value rows there are zero: the output is what the window's
    weights, of e^-nats each, leave of its (positive) values."""
    g = np.random.default_rng(seed)
    c = attention_case(seed, Hq=Hq, Hkv=Hkv, D=D, prefix=[window + 50 + 3 * i for i in range(batch)],
                       ext=[1] * batch, window=window, sinks=sinks, fp8=fp8)
    S = c["S"]
    lead = g.choice([-1.0, 1.0], size=(Hkv, D))
    first = np.concatenate([c["rtt"][r, :sinks] for r in c["rpi"]])
    k, v = 0.2 * g.standard_normal((S, Hkv, D)), 0.5 + 0.5 * np.abs(g.standard_normal((S, Hkv, D)))
    k[first], v[first] = lead * (2 * nats / np.sqrt(D)), 0.0
    q = 0.5 * np.repeat(lead, Hq // Hkv, 0) + 0.1 * g.standard_normal((batch, Hq, D))
    dead = (c["pool_k"] == (0x7F if fp8 else 0x7FFF)).all((1, 2))
    pools = [W.f32_to_bf16_bits(x.astype(np.float32)) for x in (k, v)]
    if fp8:
        pools = [oracle.fp8.quantize(x, s) for x, s in zip(pools, (c["k_scale"], c["v_scale"]))]
    for name, x in zip(("pool_k", "pool_v"), pools):
        x[dead] = 0x7F if fp8 else 0x7FFF
        c[name] = x
    c["q"] = W.f32_to_bf16_bits(q.astype(np.float32))
    return no_tiny_queries(c)


# (Hq, Hkv, D, batch, window): the groups of the e4m3 matrix path alone and in
# spans, one run a request and several; the other paths beside them
SINKS = [(8, 4, 128, 5, 200), (8, 4, 64, 5, 200), (8, 2, 128, 5, 240), (16, 4, 64, 5, 180), (8, 4, 128, 4, 1000),
         (32, 16, 64, 70, 250), (64, 16, 128, 66, 150), (4, 4, 128, 5, 200), (6, 2, 64, 5, 200), (16, 2, 128, 5, 200)]


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("nats", [6.0, 10.0, 13.0])
@pytest.mark.parametrize("shape", SINKS, ids=lambda s: f"{s[0]}q{s[1]}kv{s[2]}d_b{s[3]}_w{s[4]}")
def test_a_window_beside_a_sink_that_takes_the_weight(shape, nats, fp8):
    Hq, Hkv, D, batch, window = shape
    c = sink_case(int(nats) + window, nats, Hq=Hq, Hkv=Hkv, D=D, batch=batch, window=window, sinks=2, fp8=fp8)
    run_both(c, f"{nats} nats")
