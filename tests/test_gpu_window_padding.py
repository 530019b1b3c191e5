"""Padding rows of the sliding-window calls: a decode or extend length of 0 names
no row of req_to_token, for the calls and for their index checks."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from radixattention_prefix_shared_gb300 import binding as B  # noqa: E402
from radixattention_prefix_shared_gb300 import workloads as W  # noqa: E402

from _window import assert_within, attention_case  # noqa: E402
from test_gpu_window import Case, check_decode, decode_case  # noqa: E402

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]

DEV = "cuda:0"
NOWHERE = [-1, 2**31 - 1, -2**31]


def errors(call):
    err = torch.zeros(4, dtype=torch.int32, device=DEV)
    call(err)
    torch.cuda.synchronize()
    return err.tolist()


def set_rows(case, at):
    case.c["rpi"][at] = (NOWHERE * len(at))[: len(at)]
    case.rpi = W.int_tensor(case.c["rpi"], DEV)


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("window", [20, 900], ids=["one_run", "runs"])
def test_decode(window, fp8):
    case = decode_case(91, [0, 1500, 0, 33, 0], Hq=8, Hkv=4, D=128, window=window, sinks=2, fp8=fp8)
    set_rows(case, [0, 2, 4])
    kw = dict(max_seq_len=1500, window=window, sinks=2, pool_size=case.c["S"])
    assert errors(lambda e: B.sgl_check_decode_window_indices(case.rtt, case.rpi, case.seq, d_error=e, **kw))[0] == 0
    out = torch.full_like(case.q, 7.25)
    case.decode(out=out)
    check_decode(case, out)
    assert (out[[0, 2, 4]] == 7.25).all()
    # a live row's index and a negative length are still reported
    set_rows(case, [3])
    assert errors(lambda e: B.sgl_check_decode_window_indices(case.rtt, case.rpi, case.seq, d_error=e, **kw)) == [2, 3, 0, -1]
    seq = W.int_tensor(np.array([0, 1500, -2, 0, 0], np.int32), DEV)
    rpi = W.int_tensor(np.zeros(5, np.int32), DEV)
    assert errors(lambda e: B.sgl_check_decode_window_indices(case.rtt, rpi, seq, d_error=e, **kw)) == [3, 2, 0, -2]


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("window", [4, 700], ids=["whole", "dealt"])
def test_extend(window, fp8):
    case = Case(attention_case(92, Hq=4, Hkv=2, D=64, prefix=[0, 900, 3, 9], ext=[0, 6, 0, 3], window=window, sinks=1,
                               fp8=fp8))
    set_rows(case, [0, 2])
    kw = dict(total_extend=9, max_extend=6, max_prefix=900, window=window, sinks=1, pool_size=case.c["S"])

    def check(err, rpi=None, prefix=None):
        B.sgl_check_extend_window_indices(case.rtt, case.rpi if rpi is None else rpi,
                                          case.prefix if prefix is None else prefix, case.ext, d_error=err, **kw)
    assert errors(check)[0] == 0
    assert_within(W.bf16_bits(case.extend()), *case.want_extend(), fp8)
    bad = W.int_tensor(np.array([0, 900, -5, 9], np.int32), DEV)
    assert errors(lambda e: check(e, prefix=bad)) == [3, 2, 0, -5]
    rows = case.rpi.clone()
    rows[3] = -9
    assert errors(lambda e: check(e, rpi=rows)) == [2, 3, 0, -9]
