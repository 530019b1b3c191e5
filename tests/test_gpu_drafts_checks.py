"""Checked mode of the drafted-token calls over what the calls themselves allow."""
import pytest

torch = pytest.importorskip("torch")

from radixattention_prefix_shared_gb300 import binding as B  # noqa: E402
from radixattention_prefix_shared_gb300 import workloads as W  # noqa: E402

from _drafts import assert_attention, attention_case  # noqa: E402
from test_gpu_drafts import DEV, Case, _checked  # noqa: E402

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


def test_a_step_without_tokens():
    """All rows padding and no token: the call, the walk, the commit and the check."""
    c = attention_case(901, Hq=4, Hkv=2, D=64, prefix=[5, 60], drafts=[0, -1])
    case = Case(c)
    none = torch.zeros(0, dtype=torch.int32, device=DEV)
    case.parents, case.q = none, case.q[:0]
    assert _checked(case) == [0, 0, 0, 0]
    assert case.run().shape == case.q.shape
    rows = torch.zeros(0, 30, device=DEV)
    coins, final = torch.zeros(0, device=DEV), torch.zeros(2, device=DEV)
    path, count, token = B.sgl_verify_drafts(rows, none, none, case.drafts, coins, final, max_draft=4)
    assert (path == -1).all() and count.tolist() == [0, 0] and token.tolist() == [-1, -1]
    seq, freed, n = B.sgl_commit_drafts(case.rtt, case.rpi, case.prefix, case.drafts, none, path, count)
    assert seq.tolist() == [5, 60] and n.tolist() == [0] and freed.numel() == 0
