"""Drafted-token attention with many blocks a CTA: rings of K and V slots that go round
more than once, score, weight and output buffers used again and again, and lists of
units longer than what is listed ahead."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from _drafts_runs import MOST_STAGES, Batch  # noqa: E402

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]

# (nodes, query heads a KV head): tiles of 16, 32, 64 and 128 columns (over e4m3 pools
# the last is two tiles of 64), full and not
WIDTHS = [(3, 5), (8, 4), (13, 4), (32, 4), (29, 3)]
SHAPES = [(n, g, D, fp8) for n, g in WIDTHS for D in (64, 128) for fp8 in (False, True)]


def _blocks_a_cta(b):
    return [sum(t for _, _, t in run) for run in b.segments()]


@pytest.mark.parametrize("n,g,D,fp8", SHAPES)
def test_long_units(n, g, D, fp8):
    """Units of 30 blocks and more."""
    rng = np.random.default_rng(n)
    b = Batch(400 + n + D, Hq=8 * g, Hkv=8, D=D, prefix=[int(x) for x in rng.integers(3900, 4900, size=16)],
              drafts=[n] * 8 + [max(1, n - 2)] * 8, fp8=fp8)
    assert min(_blocks_a_cta(b)) >= 2 * MOST_STAGES
    assert max(t for run in b.segments() for _, _, t in run) > MOST_STAGES
    b.check(f"{n} nodes, {g} heads")


@pytest.mark.parametrize("n,g,D,fp8", SHAPES)
def test_units_of_a_block(n, g, D, fp8):
    """A unit a block, hundreds of requests: every block opens and ends a segment."""
    rng = np.random.default_rng(n)
    b = Batch(500 + n + D, Hq=8 * g, Hkv=8, D=D, prefix=[int(x) for x in rng.integers(0, 128 - n, size=490)],
              drafts=[int(x) for x in rng.choice([0, 1, n // 2, n, n], size=490)], fp8=fp8)
    assert min(_blocks_a_cta(b)) >= 2 * 7 and all(s == (1, 0, 1) for run in b.segments() for s in run)
    b.check(f"{n} nodes, {g} heads")


@pytest.mark.parametrize("n,g,D,fp8", SHAPES)
def test_units_of_every_length(n, g, D, fp8):
    """Units of one block to forty side by side, padding rows between them."""
    rng = np.random.default_rng(n + 1)
    prefix = [int(x) for x in np.exp(rng.uniform(0, np.log(5000), size=150))]
    b = Batch(600 + n + D, Hq=4 * g, Hkv=4, D=D, prefix=prefix, drafts=[int(x) for x in rng.choice([0, 1, 2, n], size=150)],
              fp8=fp8, kind="forest")
    kinds = {(t == nb, o == 0) for run in b.segments() for nb, o, t in run}
    assert len(kinds) >= 3  # whole units, first pieces, later ones
    b.check(f"{n} nodes, {g} heads")
