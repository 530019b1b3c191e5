"""Pins of the sliding-window and rotary oracles (closed forms, the pinned
full-causal oracle, brute force, planted slips), and the window calls' host
validation.  No GPU."""
import ctypes
import math

import numpy as np
import pytest

import oracle
from radixattention_prefix_shared_gb300 import binding as B
from radixattention_prefix_shared_gb300 import workloads as W

from _window import assert_within, attention_bound, attention_case, readers  # noqa: F401


def run_extend(c, **kw):
    a = dict(window=c["window"], sinks=c["sinks"])
    a.update(kw)
    return oracle.window.extend_attention_window(c["q"], *readers(c), c["rtt"], c["rpi"], c["prefix"], c["ext"],
                                                 c["Hkv"], a["window"], a["sinks"])


def test_visible_positions_by_enumeration():
    for P in range(12):
        for window in (1, 2, 5, 20):
            for sinks in (0, 1, 3, 20):
                want = [j for j in range(P + 1) if j < sinks or P - j < window]
                assert oracle.window.visible_positions(P, window, sinks).tolist() == want


@pytest.mark.parametrize("fp8", [False, True])
def test_a_window_over_everything_is_causal_attention(fp8):
    c = attention_case(3, Hq=4, Hkv=2, D=64, prefix=[5, 0, 9], ext=[4, 3, 0], window=100, sinks=0, fp8=fp8)
    got, _ = run_extend(c)
    if fp8:
        want = oracle.fp8.extend_attention_fp8(c["q"], c["pool_k"], c["pool_v"], c["k_scale"], c["v_scale"], c["rtt"],
                                               c["rpi"], c["prefix"], c["ext"], c["Hkv"])
    else:
        new = [c["rtt"][c["rpi"][r], p: p + e] for r, (p, e) in enumerate(zip(c["prefix"], c["ext"]))]
        new = np.concatenate(new).astype(int)
        want = oracle.extend_attention(c["q"], c["pool_k"][new], c["pool_v"][new], c["pool_k"], c["pool_v"], c["rtt"],
                                       c["rpi"], c["prefix"], c["ext"], c["Hkv"])
    assert np.abs(got - want).max() < 1e-12


def test_zero_query_gives_the_mean_of_the_visible_values():
    c = attention_case(4, Hq=2, Hkv=1, D=64, prefix=[30], ext=[6], window=7, sinks=3)
    c["q"][:] = 0
    got, _ = run_extend(c)
    V = oracle.bf16_bits_to_f64(c["pool_v"])
    for i in range(6):
        slots = [c["rtt"][c["rpi"][0], j] for j in range(31 + i) if j < 3 or j > 30 + i - 7]
        assert len(slots) == 10
        assert np.abs(got[i, 1] - V[slots, 0].mean(0)).max() < 1e-12


def test_brute_force():
    c = attention_case(5, Hq=2, Hkv=2, D=64, prefix=[9], ext=[2], window=3, sinks=1)
    got, _ = run_extend(c)
    q, K, V = (oracle.bf16_bits_to_f64(c[n]) for n in ("q", "pool_k", "pool_v"))
    for i in range(2):
        for h in range(2):
            num, den = [0.0] * 64, 0.0
            for j in range(10 + i):
                if j >= 1 and 9 + i - j >= 3:
                    continue
                s = c["rtt"][c["rpi"][0], j]
                w = math.exp(sum(q[i, h, d] * K[s, h, d] for d in range(64)) / 8.0)
                den += w
                for d in range(64):
                    num[d] += w * V[s, h, d]
            assert max(abs(num[d] / den - got[i, h, d]) for d in range(64)) < 1e-12


def test_decode_is_the_extend_of_one_token():
    c = attention_case(6, Hq=4, Hkv=2, D=64, prefix=[40, 3, 0], ext=[1, 1, 1], window=9, sinks=2)
    want, _ = run_extend(c)
    got, _ = oracle.window.decode_attention_window(c["q"], *readers(c), c["rtt"], c["rpi"], c["seq"], c["Hkv"],
                                                   c["window"], c["sinks"])
    assert np.array_equal(got, want)


@pytest.mark.parametrize("slip", [dict(window=8), dict(window=6), dict(sinks=2), dict(sinks=4)])
def test_planted_slips_exceed_the_bound(slip):
    c = attention_case(7, Hq=4, Hkv=2, D=64, prefix=[60], ext=[5], window=7, sinks=3)
    for pool in ("pool_k", "pool_v"):   # finite everywhere: the slip reads hidden rows
        dead = c[pool] == 0x7FFF
        c[pool][dead] = 0x3F80
    want, terms = run_extend(c)
    bad, _ = run_extend(c, **slip)
    assert (np.abs(bad - want) > 2 * attention_bound(want, terms, True)).any()


# ------------------------------------------------------------------ rotary positions

def test_rotation_closed_forms():
    y = np.zeros((1, 1, 64))
    y[0, 0, 0], y[0, 0, 33] = 1.0, 2.0
    f = np.zeros(32, np.float32)
    f[0], f[1] = np.float32(math.pi / 2), np.float32(math.pi)
    out, size = oracle.rope.rotate(y, [1], f)
    assert abs(out[0, 0, 32] - 1.0) < 1e-7 and abs(out[0, 0, 0]) < 1e-7      # (1, 0) a quarter turn on
    assert abs(out[0, 0, 33] + 2.0) < 1e-6 and abs(out[0, 0, 1]) < 1e-6      # (0, 2) half a turn on
    assert size[0, 0, 0] == 1.0 and size[0, 0, 1] == 2.0
    out, _ = oracle.rope.rotate(y, [1], f, interleaved=True)
    assert abs(out[0, 0, 1] - 1.0) < 1e-7 and out[0, 0, 33] == 2.0           # pair (0, 1); pair 16 unturned


def test_rotation_keeps_relative_positions():
    """q.k of rotated rows depends on the distance of their positions only."""
    g = np.random.default_rng(1)
    q, k = g.standard_normal((2, 1, 1, 64))
    f = (1e4 ** (-np.arange(32) / 32)).astype(np.float32)
    for inter in (False, True):
        dots = [float((oracle.rope.rotate(q, [a + 7], f, None, inter)[0] * oracle.rope.rotate(k, [a], f, None, inter)[0]).sum())
                for a in (0, 5, 1000)]
        assert max(dots) - min(dots) < 1e-9


def test_norm_and_axes():
    x = W.f32_to_bf16_bits(np.random.default_rng(2).standard_normal((3, 2, 64)).astype(np.float32))
    one = W.f32_to_bf16_bits(np.ones(64, np.float32))
    y, _ = oracle.rope.qk_norm_rope(x, one, 1e-12, np.zeros(3), np.zeros(0, np.float32))
    assert np.abs((y ** 2).mean(-1) - 1).max() < 1e-9
    f = np.float32([0.3] * 32)
    axis = np.array([0] * 8 + [1] * 12 + [2] * 12)
    pos = np.array([[1, 2, 3], [4, 4, 4], [0, 9, 9]])
    got, _ = oracle.rope.qk_norm_rope(x, None, 0, pos, f, axis)
    for a, sl in ((0, slice(0, 8)), (1, slice(8, 20)), (2, slice(20, 32))):
        want, _ = oracle.rope.qk_norm_rope(x, None, 0, pos[a], f)
        assert np.array_equal(got[..., sl], want[..., sl])


# ------------------------------------------------------------------ host validation

FAKE, MISALIGNED = 0x100000, 0x100008


def _dims(**kw):
    d = dict(num_q_heads=4, num_kv_heads=2, head_dim=128, pool_size=1024, sm_scale=0.0)
    d.update(kw)
    return B.make_dims(**d)


def test_decode_window_validation(cuda_lib):
    d = _dims()
    need = B.decode_window_workspace_bytes(2, 640, 100, 4, d)

    def call(fp8=False, d=d, **kw):
        a = dict(q=FAKE, pk=FAKE, pv=FAKE, ks=0.1, vs=0.1, rtt=FAKE, rows=4, stride=640, rpi=FAKE, sl=FAKE, batch=2,
                 max_s=640, window=100, sinks=4, out=FAKE, ws=FAKE, wsb=need)
        a.update(kw)
        head = (a["q"], a["pk"], a["pv"]) + ((a["ks"], a["vs"]) if fp8 else ())
        f = cuda_lib.sgl_decode_attention_window_fp8 if fp8 else cuda_lib.sgl_decode_attention_window
        return f(*head, a["rtt"], a["rows"], a["stride"], a["rpi"], a["sl"], a["batch"], a["max_s"], a["window"],
                 a["sinks"], a["out"], a["ws"], a["wsb"], ctypes.byref(d), None)
    for fp8 in (False, True):
        assert call(fp8, batch=0) == 0
        assert call(fp8, batch=-1) == 1
        assert call(fp8, window=0) == 1
        assert call(fp8, window=-5) == 1
        assert call(fp8, sinks=-1) == 1
        assert call(fp8, max_s=0) == 1
        for p in ("q", "pk", "pv", "rtt", "rpi", "sl", "out"):
            assert call(fp8, **{p: None}) == 1, p
        for p in ("q", "pk", "pv"):
            assert call(fp8, **{p: MISALIGNED}) == 1, p
        assert call(fp8, ws=None) == 3
        assert call(fp8, ws=MISALIGNED) == 3
        assert call(fp8, wsb=need - 1) == 3
        assert call(fp8, d=_dims(head_dim=96)) == 2
        assert call(fp8, d=_dims(num_q_heads=258)) == 2
    for bad in (0.0, -1.0, math.inf, math.nan):
        assert call(True, ks=bad) == 1
        assert call(True, vs=bad) == 1


def test_decode_window_workspace_is_bounded_by_the_window(cuda_lib):
    d = _dims()
    assert B.decode_window_workspace_bytes(4, 1 << 20, 512, 4, d) == B.decode_window_workspace_bytes(4, 4096, 512, 4, d)
    # the largest window and sink count do not overflow
    big = B.decode_window_workspace_bytes(4, 4096, 2**31 - 1, 2**31 - 1, d)
    assert big == B.decode_window_workspace_bytes(4, 4096, 4096, 0, d)
    assert B.decode_window_workspace_bytes(0, 4096, 512, 4, d) > 0


def test_workspaces_for_the_largest_call_serve_the_smaller(cuda_lib):
    g = np.random.default_rng(8)
    for _ in range(3000):
        hkv = int(g.choice([1, 2, 3, 4, 8, 32]))
        d = _dims(num_kv_heads=hkv, num_q_heads=hkv * int(g.choice([1, 2, 4, 5, 8, 17, 32])),
                  head_dim=int(g.choice([64, 128])))
        big = [int(np.exp(g.uniform(0, np.log(m)))) for m in (300, 1 << 17, 9000, 300)]
        small = [int(g.integers(1, m + 1)) for m in big]
        assert B.decode_window_workspace_bytes(*small, d) <= B.decode_window_workspace_bytes(*big, d), (small, big)
        # batch, total_extend, max_extend, max_prefix, window, sinks
        big = [int(np.exp(g.uniform(0, np.log(m)))) for m in (60, 20000, 4000, 30000, 9000, 300)]
        big[2] = min(big[2], big[1])
        small = [int(g.integers(1, m + 1)) for m in big]
        small[2] = min(small[2], small[1])
        assert B.extend_window_workspace_bytes(*small, d) <= B.extend_window_workspace_bytes(*big, d), (small, big)


def test_extend_window_validation(cuda_lib):
    d = _dims()
    need = B.extend_window_workspace_bytes(2, 10, 6, 30, 8, 2, d)

    def call(fp8=False, d=d, **kw):
        a = dict(q=FAKE, pk=FAKE, pv=FAKE, ks=0.1, vs=0.1, rtt=FAKE, rows=4, stride=64, rpi=FAKE, pl=FAKE, el=FAKE,
                 batch=2, total=10, max_e=6, max_p=30, window=8, sinks=2, out=FAKE, ws=FAKE, wsb=need)
        a.update(kw)
        head = (a["q"], a["pk"], a["pv"]) + ((a["ks"], a["vs"]) if fp8 else ())
        f = cuda_lib.sgl_extend_attention_window_fp8 if fp8 else cuda_lib.sgl_extend_attention_window
        return f(*head, a["rtt"], a["rows"], a["stride"], a["rpi"], a["pl"], a["el"], a["batch"], a["total"],
                 a["max_e"], a["max_p"], a["window"], a["sinks"], a["out"], a["ws"], a["wsb"], ctypes.byref(d), None)
    for fp8 in (False, True):
        assert call(fp8, batch=0) == 0
        assert call(fp8, total=0) == 0
        for kw in (dict(batch=-1), dict(total=-1), dict(max_e=-1), dict(max_p=-1), dict(window=0), dict(sinks=-1),
                   dict(max_e=11), dict(stride=0), dict(rows=0)):
            assert call(fp8, **kw) == 1, kw
        for p in ("q", "pk", "pv", "rtt", "rpi", "pl", "el", "out"):
            assert call(fp8, **{p: None}) == 1, p
        for p in ("q", "pk", "pv", "out"):
            assert call(fp8, **{p: MISALIGNED}) == 1, p
        assert call(fp8, ws=None) == 3
        assert call(fp8, wsb=need - 1) == 3
        assert call(fp8, d=_dims(head_dim=96)) == 2
        assert call(fp8, d=_dims(num_q_heads=258)) == 2
    assert call(True, ks=0.0) == 1


def test_qk_rope_validation(cuda_lib):
    d = _dims()
    Q, K, V, OUT, PK, PV = (i * 0x10000000 for i in range(1, 7))

    def call(fp8=False, d=d, **kw):
        a = dict(q=Q, qs=512, k=K, ks_=256, v=V, vs_=256, qw=FAKE, kw=FAKE, eps=1e-6, pos=FAKE, axes=1, f=FAKE,
                 ax=None, rot=128, inter=0, slots=FAKE, n=8, out=OUT, pk=PK, pv=PV, s=0.1)
        a.update(kw)
        f = cuda_lib.sgl_qk_norm_rope_store_kv_fp8 if fp8 else cuda_lib.sgl_qk_norm_rope_store_kv
        tail = (a["s"], a["s"]) if fp8 else ()
        return f(a["q"], a["qs"], a["k"], a["ks_"], a["v"], a["vs_"], a["qw"], a["kw"], a["eps"], a["pos"], a["axes"],
                 a["f"], a["ax"], a["rot"], a["inter"], a["slots"], a["n"], a["out"], a["pk"], a["pv"], *tail,
                 ctypes.byref(d), None)
    for fp8 in (False, True):
        assert call(fp8, n=0) == 0
        for kw in (dict(n=-1), dict(axes=0), dict(rot=-16), dict(rot=144), dict(inter=2), dict(eps=0.0),
                   dict(eps=math.inf), dict(eps=math.nan), dict(qs=504), dict(qs=516), dict(ks_=128), dict(vs_=260),
                   dict(axes=3)):
            assert call(fp8, **kw) == 1, kw
        assert call(fp8, rot=24) == 2
        for p in ("q", "k", "v", "pos", "f", "slots", "out", "pk", "pv"):
            assert call(fp8, **{p: None}) == 1, p
        for p in ("q", "k", "v", "out", "pk", "pv", "qw", "kw"):
            assert call(fp8, **{p: MISALIGNED}) == 1, p
        # q_out over part of what is read: q at another layout, k, v
        assert call(fp8, out=Q, qs=1024) == 1
        assert call(fp8, out=Q + 4096) == 1
        assert call(fp8, out=K + 512) == 1
        assert call(fp8, out=V - 16) == 1
        # pools over what is read, over q_out, over one another
        for kw in (dict(pk=Q), dict(pv=K), dict(pk=V), dict(pv=OUT), dict(pk=PV + 1024)):
            assert call(fp8, **kw) == 1, kw
        assert call(fp8, d=_dims(head_dim=96)) == 2
    assert call(True, s=0.0) == 1


def test_check_calls_validation(cuda_lib):
    f, g = cuda_lib.sgl_check_decode_window_indices, cuda_lib.sgl_check_extend_window_indices
    assert f(FAKE, 4, 64, FAKE, FAKE, 0, 64, 8, 2, 100, FAKE, None) == 0
    assert f(FAKE, 4, 64, FAKE, FAKE, 2, 64, 0, 2, 100, FAKE, None) == 1
    assert f(FAKE, 4, 64, FAKE, None, 2, 64, 8, 2, 100, FAKE, None) == 1
    assert f(FAKE, 4, 64, FAKE, FAKE, 2, 64, 8, 2, 100, None, None) == 1
    assert g(FAKE, 4, 64, FAKE, FAKE, FAKE, 0, 0, 0, 0, 8, 2, 100, FAKE, None) == 0
    assert g(FAKE, 4, 64, FAKE, FAKE, FAKE, 2, 4, 4, 4, 8, -1, 100, FAKE, None) == 1
    assert g(FAKE, 0, 64, FAKE, FAKE, FAKE, 2, 4, 4, 4, 8, 1, 100, FAKE, None) == 1
