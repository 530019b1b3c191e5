"""Sliding-window decodes whose lengths pass the host's maximum or the rows of
req_to_token (which positions those leave is pinned in test_window_run_host.py)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import oracle  # noqa: E402
from radixattention_prefix_shared_gb300 import workloads as W  # noqa: E402

from _window import assert_within, readers  # noqa: E402
from test_gpu_window import decode_case  # noqa: E402

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]

# (Hq, Hkv, D, lengths, window, sinks, max_seq): one run a request, several,
# rows gathered in spans; requests whose whole window lies past the maximum
SHAPES = [(8, 2, 64, [50, 60, 69, 70, 75, 300], 20, 2, 50),
          (8, 4, 128, [50, 60, 75, 300], 20, 0, 50),
          (4, 4, 128, [1500, 2100, 2600, 900], 1000, 3, 1500),
          (12, 4, 64, [700, 901] * 40, 400, 1, 600)]


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("by_rows", [False, True], ids=["max_seq_len", "rtt_stride"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"{s[0]}q{s[1]}kv{s[2]}d_w{s[4]}s{s[5]}_max{s[6]}")
def test_lengths_above_the_maximum_read_their_own_window(shape, by_rows, fp8):
    """Hidden entries of req_to_token name NaN rows, so a position that a cut
    request's query does not see would show up."""
    Hq, Hkv, D, seq, window, sinks, top = shape
    case = decode_case(top + D, seq, Hq=Hq, Hkv=Hkv, D=D, window=window, sinks=sinks, fp8=fp8)
    c = case.c
    want = oracle.window.decode_attention_window(c["q"], *readers(c), c["rtt"], c["rpi"], c["seq"], Hkv, window, sinks,
                                                 max_seq=top)
    none = np.array([n - window >= top and sinks == 0 for n in seq])
    out = torch.full_like(case.q, 5.5)
    if by_rows:
        case.rtt = case.rtt[:, :top].contiguous()
        case.decode(out=out)
    else:
        case.decode(out=out, max_seq_len=top)
    assert_within(W.bf16_bits(out), *want, fp8, rows=~none, what=str(shape))
    assert (out[torch.from_numpy(none).to(out.device)] == 5.5).all()
