"""Host maxima of the drafted-token calls that are bounds of a whole loop, not of a step."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from radixattention_prefix_shared_gb300 import binding as B  # noqa: E402
from radixattention_prefix_shared_gb300 import workloads as W  # noqa: E402

from _drafts import accept_case, assert_attention, attention_case, want_accept  # noqa: E402
from test_gpu_drafts import Case, run_accept  # noqa: E402

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("drafts", [[1], [5], [3, 0, 2]])
def test_largest_tree_above_the_steps_tokens(drafts, fp8):
    """A loop's limit of 16 or 64 nodes a tree, with fewer tokens than that in the step."""
    prefix = [300, 2, 130][: len(drafts)]
    case = Case(attention_case(320, Hq=8, Hkv=2, D=128, prefix=prefix, drafts=drafts, fp8=fp8))
    want = case.run()
    for most in (16, 64):
        assert torch.equal(case.run(max_draft=most).view(torch.int16), want.view(torch.int16))
        ws = case.new_workspace(max_draft=most)
        assert_attention(W.bf16_bits(case.run(max_draft=most, workspace=ws)), case.c)
    with pytest.raises(B.SglError) as e:
        case.run(max_draft=65)
    assert e.value.code == 2
    out = torch.full_like(case.q, 3.0)
    case.run(max_draft=16, total_draft=0, out=out)
    assert (out == 3.0).all()


def test_the_walk_takes_the_same_limits():
    c = accept_case(321, drafts=[2, 1], V=300)
    for got, w in zip(run_accept(c, max_draft=16), want_accept(c | dict(most=16))):
        assert np.array_equal(got, w)
