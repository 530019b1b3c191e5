"""A prefix that the whole batch shares, over many blocks a CTA, with references that move
and batches whose rows fill many tiles."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from _drafts_runs import Batch  # noqa: E402

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("shared,requests", [(2048, 64), (4001, 40), (130, 90)])
def test_many_rows(shared, requests, D, fp8):
    g = np.random.default_rng(shared)
    prefix = [shared + int(x) for x in g.choice([0, 1, 100, 130, 300], size=requests)]
    Batch(800 + shared, Hq=32, Hkv=8, D=D, prefix=prefix, drafts=[int(x) for x in g.choice([1, 5, 8, 8], size=requests)],
          fp8=fp8, shared=shared).check()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("D", [64, 128])
def test_scores_rise(D, fp8):
    """Shared blocks whose references move, joined with own blocks far above them."""
    step = 8.0 if fp8 else 27.0
    Batch(830, Hq=32, Hkv=8, D=D, prefix=[1600 + 37 * (i % 5) for i in range(48)], drafts=[8] * 48, fp8=fp8, step=step,
          shared=1500).check()


@pytest.mark.parametrize("fp8", [False, True])
def test_one_request_shares_with_itself(fp8):
    Batch(840, Hq=8, Hkv=2, D=128, prefix=[900], drafts=[6], fp8=fp8, shared=900).check()
    Batch(841, Hq=8, Hkv=2, D=128, prefix=[900], drafts=[6], fp8=fp8, shared=1).check()
