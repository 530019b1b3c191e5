"""Drafted-token attention whose waits give up over a workspace that held other things:
only its first 256 bytes are zero-filled, and the merge of pieces that the call did not
leave must not follow what lies behind them."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from radixattention_prefix_shared_gb300 import workloads as W  # noqa: E402

from _drafts import assert_attention, attention_case  # noqa: E402
from test_gpu_drafts import DEV, Case  # noqa: E402
from test_gpu_wait_timeout import TIMEOUT_CODE, _device_answers, short_waits  # noqa: E402

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]


def _old(words, kind):
    """What an earlier call may have left: states in fp32, codes, other integers."""
    g = torch.Generator().manual_seed(7)
    if kind == "states":
        return (torch.randn(words, generator=g) * 1e3).view(torch.int32)
    if kind == "negative":
        return torch.randint(-2**31, 0, (words,), generator=g).to(torch.int32)
    if kind == "small":  # a piece's numbers, out of order and past their ends
        return torch.randint(-3, 400, (words,), generator=g).to(torch.int32)
    return torch.full((words,), 2**31 - 1, dtype=torch.int32)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("shared", [0, 20])
@pytest.mark.parametrize("many", [False, True])
def test_over_old_contents(many, shared, fp8):
    """Few rows (a block merges one) and many (a warp does)."""
    n = [9, 4] if not many else [int(x) for x in np.random.default_rng(5).integers(1, 17, size=16)]
    prefix = [900, 30] if not many else [40 + 100 * i for i in range(16)]
    Hq = 32 if many else 8
    case = Case(attention_case(300 + shared, Hq=Hq, Hkv=2, D=128, prefix=prefix, drafts=n, shared=shared, fp8=fp8))
    assert (sum(n) * Hq > 16 * 160) == many
    ws = case.new_workspace()
    for kind in ("states", "negative", "small", "largest"):
        ws[256:].view(torch.int32).copy_(_old(ws.numel() // 4 - 64, kind).to(DEV))
        ws[:256].zero_()
        with short_waits():
            case.run(workspace=ws)
        torch.cuda.synchronize()
        assert int(ws[:4].view(torch.int32).item()) == TIMEOUT_CODE
        _device_answers()
        # the same contents under a call whose waits end
        ws[256:].view(torch.int32).copy_(_old(ws.numel() // 4 - 64, kind).to(DEV))
        ws[:256].zero_()
        assert_attention(W.bf16_bits(case.run(workspace=ws)), case.c, kind)
        assert int(ws[:4].view(torch.int32).item()) == 0
