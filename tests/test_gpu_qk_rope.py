"""Head norms, rotary positions and the KV store in one pass, against the fp64
oracle.

Bounds: bf16 outputs are rounded once, 2^-8 of the value; e4m3 codes 2^-4 of
it, or half a subnormal step (2^-10 of the scale).  In fp32 before that: the
norm's factor (the sum of D squares, the reciprocal root), the weights, the
rotation and an angle good to 2^-24 turns (sin and cos off by 2 pi 2^-24 <
2^-21) stay within 2^-18 of the pair's size |a| + |b|."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import oracle  # noqa: E402
from radixattention_prefix_shared_gb300 import binding as B  # noqa: E402
from radixattention_prefix_shared_gb300 import workloads as W  # noqa: E402

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]

DEV = "cuda:0"
EPS = 1e-6


class Case:
    def __init__(self, seed, *, n, Hq, Hkv, D, rot=None, interleaved=False, axes=1, norm=(True, True), fp8=False,
                 max_pos=5000, packed=True, theta=1e4, padding=()):
        g = np.random.default_rng(seed)
        rot = D if rot is None else rot
        self.n, self.Hq, self.Hkv, self.D, self.fp8, self.inter = n, Hq, Hkv, D, fp8, interleaved
        self.x = W.f32_to_bf16_bits((g.standard_normal((n, Hq + 2 * Hkv, D)) * 1.5).astype(np.float32))
        self.w = [W.f32_to_bf16_bits((1 + 0.2 * g.standard_normal(D)).astype(np.float32)) if on else None for on in norm]
        self.f = (theta ** (-np.arange(0, rot, 2) / max(rot, 1))).astype(np.float32)
        self.pos = g.integers(0, max_pos, size=(axes, n)).astype(np.int32)
        self.axis = g.integers(0, axes, size=rot // 2).astype(np.int32) if axes > 1 else None
        self.S = 2 * n + 5
        self.slots = g.permutation(self.S)[:n].astype(np.int32)
        for t, s in padding:
            self.slots[t] = s
        self.live = (self.slots >= 0) & (self.slots < self.S)
        self.pool = [g.integers(0, 0x7F if fp8 else 0x7F00, size=(self.S, Hkv, D)).astype(np.uint8 if fp8 else np.uint16)
                     for _ in range(2)]
        self.scales = (0.031, 0.02) if fp8 else ()
        t = W.bf16_tensor(self.x, DEV)
        q, k, v = t.split([Hq, Hkv, Hkv], dim=1)
        self.t = [q, k, v] if packed else [a.contiguous() for a in (q, k, v)]
        up = (lambda a: torch.from_numpy(a).to(DEV)) if fp8 else (lambda a: W.bf16_tensor(a, DEV))
        self.tpool = [up(a) for a in self.pool]
        self.tw = [None if w is None else W.bf16_tensor(w, DEV) for w in self.w]
        self.tf = torch.from_numpy(self.f).to(DEV) if rot else None
        self.tpos = W.int_tensor(self.pos if axes > 1 else self.pos[0], DEV) if rot else None
        self.taxis = None if self.axis is None else W.int_tensor(self.axis, DEV)
        self.tslots = W.int_tensor(self.slots, DEV)

    def run(self, **kw):
        f = B.sgl_qk_norm_rope_store_kv_fp8 if self.fp8 else B.sgl_qk_norm_rope_store_kv
        return f(*self.t, self.tpos, self.tf, self.tslots, *self.tpool, *self.scales, q_weight=self.tw[0],
                 k_weight=self.tw[1], eps=EPS, freq_axis=self.taxis, interleaved=self.inter, **kw)

    def check(self, q_out):
        Hq, Hkv, live = self.Hq, self.Hkv, self.live
        pos = self.pos if self.pos.shape[0] > 1 else self.pos[0]
        want_q, size_q = oracle.rope.qk_norm_rope(self.x[:, :Hq], self.w[0], EPS, pos, self.f, self.axis, self.inter)
        want_k, size_k = oracle.rope.qk_norm_rope(self.x[:, Hq: Hq + Hkv], self.w[1], EPS, pos, self.f, self.axis,
                                                  self.inter)
        got_q = oracle.bf16_bits_to_f64(W.bf16_bits(q_out))
        bound = 2.0 ** -8 * np.abs(want_q) + 2.0 ** -18 * size_q
        assert (np.abs(got_q - want_q)[live] <= bound[live]).all(), "q"
        rest = np.setdiff1d(np.arange(self.S), self.slots[live])
        at = self.slots[live]
        if self.fp8:
            pools = [p.cpu().numpy() for p in self.tpool]
            ks, vs = self.scales
            got_k = oracle.fp8.e4m3_decode(pools[0][at]) * ks
            top = 448 * ks
            want = np.clip(want_k[live], -top, top)
            bound = 2.0 ** -4 * np.abs(want) + 2.0 ** -10 * ks + 2.0 ** -18 * size_k[live]
            assert np.array_equal(pools[1][at], oracle.fp8.quantize(self.x[live][:, Hq + Hkv:], vs)), "v codes"
        else:
            pools = [W.bf16_bits(p) for p in self.tpool]
            got_k, want = oracle.bf16_bits_to_f64(pools[0][at]), want_k[live]
            bound = 2.0 ** -8 * np.abs(want) + 2.0 ** -18 * size_k[live]
            assert np.array_equal(pools[1][at], self.x[live][:, Hq + Hkv:]), "v rows"
        assert (np.abs(got_k - want) <= bound).all(), "k"
        for i in range(2):
            assert np.array_equal(pools[i][rest], self.pool[i][rest]), "rows of other slots"


SHAPES = [
    dict(n=1, Hq=1, Hkv=1, D=64),
    dict(n=1, Hq=16, Hkv=8, D=128),
    dict(n=64, Hq=16, Hkv=8, D=128),
    dict(n=77, Hq=32, Hkv=8, D=128, rot=64),
    dict(n=33, Hq=5, Hkv=5, D=64, rot=16),
    dict(n=130, Hq=6, Hkv=3, D=64, rot=48),
    dict(n=40, Hq=12, Hkv=1, D=128, rot=96),
    dict(n=31, Hq=7, Hkv=1, D=128, rot=0),
    dict(n=301, Hq=4, Hkv=4, D=64, axes=3),
    dict(n=50, Hq=8, Hkv=2, D=128, axes=2, rot=112),
    dict(n=5000, Hq=3, Hkv=1, D=64),
]


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("interleaved", [False, True], ids=["halves", "adjacent"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "_".join(f"{k}{v}" for k, v in s.items()))
def test_matches_oracle(shape, interleaved, fp8):
    c = Case(shape["n"] + shape["D"], interleaved=interleaved, fp8=fp8, **shape)
    c.check(c.run())


@pytest.mark.parametrize("norm", [(False, False), (True, False), (False, True)])
def test_norms_are_optional(norm):
    c = Case(5, n=45, Hq=4, Hkv=2, D=128, norm=norm)
    c.check(c.run())
    c = Case(6, n=45, Hq=4, Hkv=2, D=64, norm=norm, fp8=True, packed=False)
    c.check(c.run())


def test_far_and_negative_positions():
    """Angles stay exact where a float32 product would be off by radians."""
    c = Case(7, n=64, Hq=2, Hkv=2, D=128)
    c.pos[0, :8] = [2**31 - 1, -2**31, -1, 1 << 20, (1 << 24) + 1, -(1 << 20), 0, 123456789]
    c.tpos = W.int_tensor(c.pos[0], DEV)
    c.check(c.run())


def test_padding_tokens_leave_everything_alone():
    for fp8 in (False, True):
        c = Case(8, n=20, Hq=4, Hkv=2, D=64, fp8=fp8, padding=[(0, -1), (7, 45), (19, 2**31 - 1), (3, -2**31)])
        out = torch.full((20, 4, 64), 9.5, dtype=torch.bfloat16, device=DEV)
        c.check(c.run(q_out=out))
        assert (out[[0, 3, 7, 19]] == 9.5).all()


def test_in_place_queries():
    c = Case(9, n=37, Hq=4, Hkv=2, D=128, packed=False)
    out = c.run(q_out=c.t[0])
    assert out.data_ptr() == c.t[0].data_ptr()
    c.check(out)
    c = Case(9, n=37, Hq=4, Hkv=2, D=128)
    with pytest.raises(B.SglError):       # over the packed projection's own rows
        c.run(q_out=torch.as_strided(c.t[0], (37, 4, 128), (512, 128, 1)))


def test_zero_rows_and_large_values():
    c = Case(10, n=12, Hq=2, Hkv=2, D=64)
    c.x[:4] = 0
    c.x[4:8, :, ::3] = 0x7F00             # 1.7e38: their squares overflow to a norm factor of 0
    t = W.bf16_tensor(c.x, DEV)
    c.t = list(t.split([2, 2, 2], dim=1))
    out = oracle.bf16_bits_to_f64(W.bf16_bits(c.run()))
    assert (out[:4] == 0).all() and np.isfinite(out).all()


def test_no_tokens():
    c = Case(11, n=3, Hq=2, Hkv=2, D=64)
    c.t = [a[:0] for a in c.t]
    c.tslots, c.tpos = c.tslots[:0], c.tpos[:0]
    assert c.run().shape == (0, 2, 64)


def test_stored_rows_are_what_the_store_writes():
    """Without norm and rotation the call is sgl_store_kv(_fp8), bit for bit."""
    for fp8 in (False, True):
        c = Case(12, n=70, Hq=4, Hkv=2, D=128, rot=0, norm=(False, False), fp8=fp8)
        want = [p.clone() for p in c.tpool]
        c.run()
        store = B.sgl_store_kv_fp8 if fp8 else B.sgl_store_kv
        store(c.t[1].contiguous(), c.t[2].contiguous(), c.tslots, *want, *c.scales)
        torch.cuda.synchronize()
        for a, b in zip(c.tpool, want):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("scale", [1.0, 0.0173, 1 / 3, 0.031, 7.77, 2.0**-60, 3e-20, 2.0**61, 1e-40, 3e38])
def test_codes_of_every_bf16_value(scale):
    """Every finite bf16 value over the scale: the codes of sgl_store_kv_fp8, bit for bit."""
    bits = np.arange(1 << 16, dtype=np.uint32).astype(np.uint16)
    bits = bits[(bits & 0x7F80) != 0x7F80]
    rows = np.zeros((512, 1, 128), np.uint16)
    rows.reshape(-1)[: bits.size] = bits
    x = W.bf16_tensor(rows, DEV)
    slots = torch.arange(512, dtype=torch.int32, device=DEV)
    got = [torch.zeros(512, 1, 128, dtype=torch.uint8, device=DEV) for _ in range(2)]
    want = [torch.zeros_like(p) for p in got]
    B.sgl_qk_norm_rope_store_kv_fp8(x, x, x, None, None, slots, *got, scale, scale)
    B.sgl_store_kv_fp8(x, x, slots, *want, scale, scale)
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_binding_refuses_what_it_would_misread():
    c = Case(13, n=9, Hq=4, Hkv=2, D=64)
    for i, bad in ((0, c.t[0].transpose(1, 2)), (1, c.t[1][:, :1]), (2, c.t[2].float()), (0, c.t[0].cpu())):
        keep = c.t[i]
        c.t[i] = bad
        with pytest.raises(ValueError):
            c.run()
        c.t[i] = keep
    for attr, bad in (("tslots", c.tslots.long()), ("tpos", c.tpos[:4]), ("tf", c.tf.double()),
                      ("tslots", c.tslots[:8])):
        keep = getattr(c, attr)
        setattr(c, attr, bad)
        with pytest.raises(ValueError):
            c.run()
        setattr(c, attr, keep)
