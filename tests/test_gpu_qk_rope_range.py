"""Head norms over the whole range of bf16: rows whose squares overflow, or
underflow beside eps, beside ordinary rows of the same warp, within the bounds
of test_gpu_qk_rope.py (whose 2^-18 of a pair's size covers the norm's
factor wherever the row lies: from 2^126 on it is an fp32 subnormal, below 2^-126,
but above 2^-128.5 and so good to 2^-150 / 2^-128.5 < 2^-21).

A value of 1 in a row of 3e38 comes out at 4e-39, below bf16's smallest normal
value of 2^-126: there a rounding is off by half of bf16's smallest step, 2^-134,
whatever the value's size (45 steps of 2^-133 are 1.1% apart, half of which is
above 2^-8 of the value).  `check` adds that."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import oracle  # noqa: E402
from radixattention_prefix_shared_gb300 import workloads as W  # noqa: E402

from test_gpu_qk_rope import DEV, EPS, Case  # noqa: E402

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]


def set_rows(c, x):
    """The case's projection becomes x [n, Hq + 2 Hkv, D]; its V rows stay."""
    Hkv = c.Hkv
    keep = c.x[:, -Hkv:].copy()
    c.x = W.f32_to_bf16_bits(x.astype(np.float32))
    assert ((c.x & 0x7F80) != 0x7F80).all()      # finite
    c.x[:, -Hkv:] = keep
    c.t = list(W.bf16_tensor(c.x, DEV).split([c.Hq, Hkv, Hkv], dim=1))


def check(c, q_out):
    """The rows of a bf16 case, half a subnormal step of bf16 allowed."""
    for rows, w, got in ((slice(0, c.Hq), c.w[0], W.bf16_bits(q_out)),
                         (slice(c.Hq, c.Hq + c.Hkv), c.w[1], W.bf16_bits(c.tpool[0])[c.slots])):
        want, size = oracle.rope.qk_norm_rope(c.x[:, rows], w, EPS, c.pos[0], c.f, None, c.inter)
        bound = 2.0 ** -8 * np.abs(want) + 2.0 ** -18 * size + 2.0 ** -134
        assert (np.abs(oracle.bf16_bits_to_f64(got) - want) <= bound).all()


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("interleaved", [False, True], ids=["halves", "adjacent"])
@pytest.mark.parametrize("D", [64, 128])
def test_rows_of_every_size(D, interleaved, fp8):
    c = Case(D, n=90, Hq=6, Hkv=3, D=D, interleaved=interleaved, fp8=fp8)
    g = np.random.default_rng(D)
    # from 2^-20 to where the largest of D normal values still is a bf16
    size = 2.0 ** g.uniform(-20, 125, size=(90, 12, 1))
    set_rows(c, np.clip(g.standard_normal((90, 12, D)), -7, 7) * size)
    c.check(c.run())


@pytest.mark.parametrize("interleaved", [False, True], ids=["halves", "adjacent"])
@pytest.mark.parametrize("D", [64, 128])
def test_pairs_of_the_largest_values(D, interleaved):
    """Both values of a pair near the top, turned by 45 degrees: their sum before
    the norm's factor is past fp32."""
    c = Case(3, n=16, Hq=2, Hkv=2, D=D, interleaved=interleaved, norm=(True, True))
    c.f[:] = np.float32(np.pi / 4)
    c.tf = torch.from_numpy(c.f).to(DEV)
    c.pos[0] = np.arange(16)
    c.tpos = W.int_tensor(c.pos[0], DEV)
    top = 3.38e38
    x = np.full((16, 6, D), top)
    x[:, 1::2] *= np.where(np.arange(D) % 3 == 0, -1, 1)
    x[5:8, :, ::2] = 1.0
    x[8, :, 1:] = 0                       # one value that takes the row
    x[9:12] *= 2.0 ** -67                 # the sum of squares just past, just below and at the end of fp32
    x[12] *= 2.0 ** -68
    set_rows(c, x)
    check(c, c.run())


def far_rows(c, g, share):
    """A share of the case's rows at 2^90 to 2^120 of their size."""
    x = oracle.bf16_bits_to_f64(c.x)
    up = g.uniform(size=x.shape[:2] + (1,)) < share
    set_rows(c, np.where(up, x * 2.0 ** np.floor(g.uniform(90, 120, size=up.shape)), x))


@pytest.mark.parametrize("shape", [dict(n=9000, Hq=3, Hkv=1, D=64), dict(n=6000, Hq=6, Hkv=2, D=128),
                                   dict(n=700, Hq=36, Hkv=9, D=64), dict(n=1, Hq=16, Hkv=8, D=128),
                                   dict(n=40, Hq=70, Hkv=35, D=128, rot=64)],
                         ids=lambda s: "_".join(f"{k}{v}" for k, v in s.items()))
@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
def test_a_few_far_rows_among_many(shape, fp8):
    """Warps with several tokens, tokens dealt to several warps, padding."""
    c = Case(21, fp8=fp8, padding=[(0, -1), (7, 2**31 - 1)] if shape["n"] > 7 else (), **shape)
    far_rows(c, np.random.default_rng(22), 0.01 if shape["n"] > 100 else 0.3)
    out = torch.full((c.n, c.Hq, c.D), 2.5, dtype=torch.bfloat16, device=DEV)
    c.check(c.run(q_out=out))
    assert (out[torch.from_numpy(~c.live).to(DEV)] == 2.5).all()


@pytest.mark.parametrize("norm", [(True, False), (False, True)])
def test_one_norm_and_queries_in_place(norm):
    """Rows without a weight are not the norm's to scale; q_out over q."""
    c = Case(23, n=300, Hq=6, Hkv=2, D=128, norm=norm, packed=False)
    x = oracle.bf16_bits_to_f64(c.x)
    rows = slice(0, 6) if norm[0] else slice(6, 8)
    x[::5, rows] *= 2.0 ** 100
    set_rows(c, x)
    c.t = [t.contiguous() for t in c.t]
    out = c.run(q_out=c.t[0])
    assert out.data_ptr() == c.t[0].data_ptr()
    c.check(out)


def test_rows_that_are_not_finite_spoil_no_others():
    """A NaN makes its row NaN; beside an infinity the rest of its row is 0."""
    c = Case(24, n=50, Hq=4, Hkv=2, D=64)
    clean = c.run().clone()
    pool = [p.clone() for p in c.tpool]
    c.x[3, 0, 10], c.x[9, 5, 0], c.x[30, 2, 63] = 0x7FC0, 0x7FC0, 0x7F80
    c.t = list(W.bf16_tensor(c.x, DEV).split([4, 2, 2], dim=1))
    out = c.run()
    assert torch.isnan(out[3, 0]).all() and torch.isnan(c.tpool[0][int(c.slots[9]), 1]).all()
    assert torch.isnan(out[30, 2, [31, 63]]).all()        # the infinity over itself, and its pair
    assert (out[30, 2, :31] == 0).all() and (out[30, 2, 32:63] == 0).all()
    keep = torch.ones(50, 4, dtype=torch.bool, device=DEV)
    keep[3, 0] = keep[30, 2] = False
    assert torch.equal(out[keep], clean[keep])
    rows = torch.ones(c.S, 2, dtype=torch.bool, device=DEV)
    rows[int(c.slots[9]), 1] = False
    assert torch.equal(c.tpool[0][rows], pool[0][rows])
