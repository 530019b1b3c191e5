"""Memory of the sliding-window calls on a stream of the caller's choice: what
the caller drops, and what a call makes for itself, is not handed out again
while the stream still works on it."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from radixattention_prefix_shared_gb300 import binding as B  # noqa: E402
from radixattention_prefix_shared_gb300 import workloads as W  # noqa: E402

from _window import assert_within, attention_case  # noqa: E402
from test_gpu_qk_rope import Case as RopeCase  # noqa: E402
from test_gpu_window import Case, check_decode, decode_case  # noqa: E402

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]

DEV = "cuda:0"


class Busy:
    """A stream with some 60 ms of products ahead of what is launched next."""

    def __init__(self, stream=None):
        self.stream = torch.cuda.Stream() if stream is None else stream
        self.a = torch.randn(8192, 8192, device=DEV, dtype=torch.bfloat16)
        self.b = torch.empty_like(self.a)
        # (the first product, fill or event of a process waits for its set-up, and
        # a new segment may wait for the device: both are taken here)
        self.fill(1)
        for n in (200, 3 << 20, 30 << 20):
            torch.zeros(n, dtype=torch.uint8, device=DEV)
        torch.zeros(9, device=DEV).record_stream(self.stream)
        torch.cuda.synchronize()

    def fill(self, n=100):
        with torch.cuda.stream(self.stream):
            for _ in range(n):
                torch.mm(self.a, self.a, out=self.b)


def taken(tensors):
    """Storage addresses and sizes of tensors that are about to be dropped."""
    return [(t.untyped_storage().data_ptr(), t.untyped_storage().nbytes()) for t in tensors if t is not None]


def claim(memory, keep, busy):
    """Allocates and overwrites the sizes just dropped, several times each;
    what came back.  (Zeros: an index read there stays in range.)"""
    new = [torch.zeros(n, dtype=torch.uint8, device=DEV) for _, n in memory for _ in range(4)]
    keep += new
    assert not busy.stream.query(), "the stream was done before the memory could be asked for"
    return sorted({p for p, _ in memory} & {t.untyped_storage().data_ptr() for t in new})


@pytest.mark.parametrize("handle", [False, True], ids=["stream", "handle"])
@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
def test_dropped_inputs_of_the_norm_and_store(fp8, handle):
    busy, keep = Busy(), []
    RopeCase(79, n=9, Hq=8, Hkv=2, D=128, axes=3, fp8=fp8).run()     # (the kernels' set-up)
    c = RopeCase(80, n=900, Hq=8, Hkv=2, D=128, axes=3, fp8=fp8)
    torch.cuda.synchronize()
    busy.fill()
    out = c.run(stream=busy.stream.cuda_stream if handle else busy.stream)
    memory = taken([c.t[0], *c.tw, c.tf, c.tpos, c.taxis, c.tslots])
    c.t = c.tw = c.tf = c.tpos = c.taxis = c.tslots = None
    assert claim(memory, keep, busy) == []
    torch.cuda.synchronize()
    c.check(out)


@pytest.mark.parametrize("handle", [False, True], ids=["stream", "handle"])
@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("kind", ["decode", "extend"])
def test_dropped_inputs_of_the_attention(kind, fp8, handle):
    busy, keep = Busy(), []
    if kind == "decode":
        case = decode_case(81, [3000, 40, 900], Hq=8, Hkv=4, D=128, window=2000, sinks=4, fp8=fp8)
        want = None
    else:
        case = Case(attention_case(82, Hq=8, Hkv=4, D=128, prefix=[900, 3], ext=[30, 40], window=500, sinks=4, fp8=fp8))
        want = case.want_extend()
    getattr(case, kind)()                                            # (the kernels' set-up)
    torch.cuda.synchronize()
    busy.fill()
    out = getattr(case, kind)(stream=busy.stream.cuda_stream if handle else busy.stream)
    names = ["q", "pk", "pv", "rtt", "rpi", "prefix", "ext", "seq"]
    unread = {"decode": ["prefix", "ext"], "extend": ["seq"]}[kind]
    memory = taken([getattr(case, n) for n in names if n not in unread])
    for n in names:
        setattr(case, n, None)
    assert claim(memory, keep, busy) == []
    torch.cuda.synchronize()
    if want is None:
        check_decode(case, out)
    else:
        assert_within(W.bf16_bits(out), *want, fp8)


def test_dropped_inputs_of_the_checks():
    busy, keep = Busy(), []
    case = Case(attention_case(83, Hq=2, Hkv=2, D=64, prefix=[40, 0], ext=[6, 4], window=8, sinks=3))
    err = torch.zeros(4, dtype=torch.int32, device=DEV)
    B.sgl_check_decode_window_indices(case.rtt, case.rpi, case.seq, max_seq_len=46, window=8, sinks=3,
                                      pool_size=case.c["S"], d_error=err)
    torch.cuda.synchronize()
    busy.fill()
    B.sgl_check_decode_window_indices(case.rtt, case.rpi, case.seq, max_seq_len=46, window=8, sinks=3,
                                      pool_size=case.c["S"], d_error=err, stream=busy.stream)
    B.sgl_check_extend_window_indices(case.rtt, case.rpi, case.prefix, case.ext, total_extend=10, max_extend=6,
                                      max_prefix=40, window=8, sinks=3, pool_size=case.c["S"], d_error=err,
                                      stream=busy.stream)
    memory = taken([case.rtt, case.rpi, case.prefix, case.ext, case.seq])
    case.rtt = case.rpi = case.prefix = case.ext = case.seq = None
    assert claim(memory, keep, busy) == []
    torch.cuda.synchronize()
    assert err.tolist() == [0, 0, 0, 0]


def test_handle_of_the_default_stream():
    """Handle 0 is the default stream, for the call and for what it allocates."""
    assert B._stream_object(0) == torch.cuda.default_stream()
    side = torch.cuda.Stream()
    assert B._stream_object(side.cuda_stream).cuda_stream == side.cuda_stream and B._stream_object(side) is side
    case = decode_case(84, [3000, 900], Hq=8, Hkv=4, D=128, window=2000, sinks=4)
    case.decode()
    busy = Busy(torch.cuda.default_stream())
    busy.fill()
    with torch.cuda.stream(side):            # the call's own buffers are the default stream's
        out = case.decode(stream=0)
        ptr = out.untyped_storage().data_ptr()
        keep = [torch.zeros_like(out) for _ in range(8)]
        assert not busy.stream.query() and ptr not in {t.untyped_storage().data_ptr() for t in keep}
    torch.cuda.synchronize()
    check_decode(case, out)


def test_captured_on_its_own_stream():
    """``stream=`` naming the capturing stream: the graph replays, and the memory
    it was given stays its own."""
    case = decode_case(85, [3000, 900], Hq=8, Hkv=4, D=128, window=2000, sinks=4)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        case.decode(stream=side)
        side.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            out = case.decode(stream=side)
    for _ in range(3):
        torch.full((1 << 22,), np.nan, device=DEV)
        out.fill_(0)
        g.replay()
        torch.cuda.synchronize()
        check_decode(case, out)
