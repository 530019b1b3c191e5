"""Drafted-token attention whose references move inside a CTA's run of blocks: the
scores rise from block to block and are largest in the last one, or a unit's first
block hides keys, so that the reference is set again in the next."""
import pytest

torch = pytest.importorskip("torch")

from _drafts_runs import Batch  # noqa: E402

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]

# nodes a request with four query heads a KV head: every width of a tile, and two tiles over e4m3 pools
WIDTHS = [4, 8, 16, 32]


def _last_blocks(b):
    """Segments of several blocks that end with their unit's last one."""
    return [s for run in b.segments() for s in run if s[2] >= 2 and s[1] + s[2] == s[0]]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n", WIDTHS)
def test_scores_rise_to_the_last_block(n, D, fp8):
    """A weight may exceed its reference by 2^30 (e4m3 pools: 2^7): every block after a
    segment's first moves it, the one with the tree too."""
    step, least = (8.0, 5.0) if fp8 else (27.0, 21.0)
    b = Batch(100 + n, Hq=32, Hkv=8, D=D, prefix=[1500, 1411, 1290, 1535, 1400, 1472], drafts=[n] * 6, fp8=fp8,
              step=step)
    assert len(_last_blocks(b)) >= 10 and max(t for run in b.segments() for _, _, t in run) >= 3
    for r in (0, 3):
        s, _ = b.scores(r, 5)
        tops = torch.stack([s[..., i: i + 128].amax(-1) for i in range(0, s.shape[-1], 128)])
        tops = tops[: 1 + (b.prefix[r] - 1) // 128]
        assert float((tops[1:] - tops[:-1]).min()) > least
    b.check(f"{n} nodes")


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n,g", [(16, 1), (16, 2), (32, 2), (64, 2)])
def test_first_blocks_that_hide_keys(n, g, D, fp8):
    """Trees that begin in a unit's first block and end in its second."""
    prefix = [128 - n + 1 + (7 * i) % (n - 1) for i in range(60)]
    b = Batch(200 + n + g, Hq=4 * g, Hkv=4, D=D, prefix=prefix, drafts=[n] * 60, fp8=fp8, std=1.5)
    assert sum(s == (2, 0, 2) for run in b.segments() for s in run) >= 40
    b.check(f"{n} nodes, {g} heads")
