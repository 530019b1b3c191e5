"""Checked mode of the drafted-token calls over what the calls themselves allow."""
import pytest

torch = pytest.importorskip("torch")

from radixattention_prefix_shared_gb300 import workloads as W  # noqa: E402

from _drafts import assert_attention, attention_case  # noqa: E402
from test_gpu_drafts import Case, _checked  # noqa: E402

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]


def test_padding_rows_of_any_kind():
    """A draft_lens entry of 0 or less: nothing of the request is read, or reported."""
    c = attention_case(900, Hq=4, Hkv=2, D=64, prefix=[40, 3, 50, 3], drafts=[4, -1, 3, -5], shared=30)
    c["prefix"][[1, 3]] = [-9, 2**30]
    case = Case(c)
    kw = dict(max_prefix=50)
    assert _checked(case, **kw) == [0, 0, 0, 0]
    assert_attention(W.bf16_bits(case.run(**kw)), c)
    assert _checked(case, total_draft=6, **kw)[0] == 5
    bad = Case(c)
    bad.parents[4] = 1   # the second request's first node
    assert _checked(bad, **kw) == [11, 2, 0, 1]
