"""Host values of the sliding-window calls that an int32 does not hold: refused,
where ctypes would cut them to another window or length."""
import sys

import pytest

torch = pytest.importorskip("torch")

from radixattention_prefix_shared_gb300 import binding as B  # noqa: E402

BAD = [2**31, 2**32 + 5, -2**31, -2**32 + 7, sys.maxsize]


def dims():
    return B.make_dims(8, 4, 128, 1000)


@pytest.mark.parametrize("bad", BAD)
def test_sizes(bad):
    good = dict(batch=4, max_seq_len=3000, window=2000, sinks=4)
    for arg in good:
        with pytest.raises(ValueError, match=arg):
            B.decode_window_workspace_bytes(**dict(good, **{arg: bad}), dims=dims())
    good = dict(batch=4, total_extend=90, max_extend=60, max_prefix=900, window=700, sinks=4)
    for arg in good:
        with pytest.raises(ValueError, match=arg):
            B.extend_window_workspace_bytes(**dict(good, **{arg: bad}), dims=dims())
    assert B.decode_window_workspace_bytes(4, 2**31 - 1, 2**31 - 1, 2**31 - 1, dims()) > 256


@pytest.mark.gpu
@pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")
@pytest.mark.parametrize("bad", BAD)
def test_calls(bad):
    from _window import attention_case
    from test_gpu_window import Case
    case = Case(attention_case(90, Hq=4, Hkv=2, D=64, prefix=[9, 30], ext=[1, 1], window=4, sinks=1))
    for arg in ("window", "sinks", "max_seq_len"):
        with pytest.raises(ValueError, match=arg):
            case.decode(**{arg: bad})
    for arg in ("window", "sinks", "max_extend", "max_prefix", "total_extend"):
        with pytest.raises(ValueError, match=arg):
            case.extend(**{arg: bad})
    err = torch.zeros(4, dtype=torch.int32, device="cuda:0")
    kw = dict(window=4, sinks=1, pool_size=case.c["S"], d_error=err)
    for arg in ("window", "sinks", "max_seq_len"):
        with pytest.raises(ValueError, match=arg):
            B.sgl_check_decode_window_indices(case.rtt, case.rpi, case.seq, **(kw | dict(max_seq_len=31) | {arg: bad}))
    ext = dict(kw, total_extend=2, max_extend=1, max_prefix=30)
    for arg in ("window", "sinks", "max_extend", "max_prefix", "total_extend"):
        with pytest.raises(ValueError, match=arg):
            B.sgl_check_extend_window_indices(case.rtt, case.rpi, case.prefix, case.ext, **(ext | {arg: bad}))
