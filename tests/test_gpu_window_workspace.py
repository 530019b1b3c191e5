"""One workspace for the sliding-window decodes and extends of a step: the
extend's wait status, its first word, is set by the extend alone."""
import pytest

torch = pytest.importorskip("torch")

from radixattention_prefix_shared_gb300 import binding as B  # noqa: E402
from radixattention_prefix_shared_gb300 import workloads as W  # noqa: E402

from _window import assert_within, attention_case  # noqa: E402
from test_gpu_window import Case, check_decode, decode_case  # noqa: E402

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]

DEV = "cuda:0"


def head(ws):
    return ws[:256].cpu()


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("heads", [(8, 4, 128), (4, 4, 64), (3, 1, 128)], ids=str)
def test_a_shared_workspace_keeps_the_status_word(heads, fp8):
    Hq, Hkv, D = heads
    dec = decode_case(70, [3000, 900, 0, 2049], Hq=Hq, Hkv=Hkv, D=D, window=2048, sinks=4, fp8=fp8)
    ext = Case(attention_case(71, Hq=Hq, Hkv=Hkv, D=D, prefix=[900, 30], ext=[60, 9], window=700, sinks=4, fp8=fp8))
    dims = B.make_dims(Hq, Hkv, D, dec.c["S"])
    nbytes = max(B.decode_window_workspace_bytes(4, 3000, 2048, 4, dims),
                 B.extend_window_workspace_bytes(2, 69, 60, 900, 700, 4, dims))
    ws = B.new_workspace(nbytes, DEV)
    for _ in range(2):
        check_decode(dec, dec.decode(workspace=ws))          # several runs a request: states are written
        assert not head(ws).any(), "decode wrote over the status word"
        assert_within(W.bf16_bits(ext.extend(workspace=ws)), *ext.want_extend(), fp8)
        assert not head(ws).any()
    # a status that an extend left outlasts the decodes behind it
    ws[:4] = torch.tensor([1, 0x57, 0, 0], dtype=torch.uint8)
    dec.decode(workspace=ws)
    assert head(ws)[:4].tolist() == [1, 0x57, 0, 0] and not head(ws)[4:].any()


def test_the_smallest_workspace_holds_the_states_behind_the_status():
    """A buffer of exactly the size asked for: nothing is written past it."""
    for Hq, Hkv, D, lens, window in ((8, 4, 128, [3000, 2500], 2048), (2, 1, 64, [5000], 4096), (4, 4, 64, [9], 8)):
        dec = decode_case(72, lens, Hq=Hq, Hkv=Hkv, D=D, window=window, sinks=2)
        need = B.decode_window_workspace_bytes(len(lens), max(lens), window, 2, B.make_dims(Hq, Hkv, D, dec.c["S"]))
        buf = torch.full((need + 4096,), 0xA5, dtype=torch.uint8, device=DEV)
        check_decode(dec, dec.decode(workspace=buf[:need]))
        assert (buf[need:] == 0xA5).all() and (buf[:256] == 0xA5).all()
