"""The sliding-window operators as a serving step uses them: norm + rotation +
store, then the attention over what was stored -- in order on one stream, on
other streams, in captured graphs, and with bounded waits that give up."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import oracle  # noqa: E402
from radixattention_prefix_shared_gb300 import binding as B  # noqa: E402
from radixattention_prefix_shared_gb300 import workloads as W  # noqa: E402

from _window import assert_within, attention_case  # noqa: E402
from test_gpu_qk_rope import Case as RopeCase  # noqa: E402
from test_gpu_wait_timeout import TIMEOUT_CODE, short_waits  # noqa: E402
from test_gpu_window import Case, check_decode, decode_case  # noqa: E402

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]

DEV = "cuda:0"


class Layer:
    """One layer's step of a batch: chunks of new tokens, then single tokens."""

    def __init__(self, seed, fp8, *, Hq=8, Hkv=4, D=128, window=40, sinks=3, prefix=(0, 70, 5), ext=(50, 9, 33),
                 steps=4):
        g = np.random.default_rng(seed)
        self.g, self.fp8, self.Hq, self.Hkv, self.D, self.window, self.sinks = g, fp8, Hq, Hkv, D, window, sinks
        self.scales = (0.05, 0.03) if fp8 else ()
        n = len(ext)
        self.lens = np.array(prefix, np.int64)
        total = sum(prefix) + sum(ext) + n * steps
        self.S = total + 9
        perm = g.permutation(self.S).astype(np.int32)
        self.rtt = np.full((n + 1, max(prefix) + max(ext) + steps + 3), perm[-1], np.int32)
        self.rows, at = g.permutation(n + 1)[:n].astype(np.int32), 0
        for r in range(n):
            m = prefix[r] + ext[r] + steps
            self.rtt[self.rows[r], :m] = perm[at: at + m]
            at += m
        self.pk, self.pv = (torch.zeros(self.S, Hkv, D, dtype=torch.uint8 if fp8 else torch.bfloat16, device=DEV)
                            for _ in range(2))
        self.w = [W.bf16_tensor(W.f32_to_bf16_bits((1 + 0.1 * g.standard_normal(D)).astype(np.float32)), DEV)
                  for _ in range(2)]
        self.f = torch.from_numpy((1e4 ** (-np.arange(0, D, 2) / D)).astype(np.float32)).to(DEV)
        self.trtt, self.trows = W.int_tensor(self.rtt, DEV), W.int_tensor(self.rows, DEV)
        if sum(prefix):   # what earlier steps stored
            self.store(list(prefix), np.zeros(n, np.int64))

    def qkv(self, tokens):
        x = self.g.standard_normal((tokens, self.Hq + 2 * self.Hkv, self.D)).astype(np.float32)
        return W.bf16_tensor(W.f32_to_bf16_bits(x), DEV)

    def positions(self, new, start):
        pos = np.concatenate([np.arange(s, s + m) for s, m in zip(start, new)]).astype(np.int32)
        slots = np.concatenate([self.rtt[r, s: s + m] for r, s, m in zip(self.rows, start, new)]).astype(np.int32)
        return W.int_tensor(pos, DEV), W.int_tensor(slots, DEV)

    def store(self, new, start, x=None, **kw):
        x = self.qkv(sum(new)) if x is None else x
        pos, slots = self.positions(new, start)
        f = B.sgl_qk_norm_rope_store_kv_fp8 if self.fp8 else B.sgl_qk_norm_rope_store_kv
        return f(*x.split([self.Hq, self.Hkv, self.Hkv], 1), pos, self.f, slots, self.pk, self.pv, *self.scales,
                 q_weight=self.w[0], k_weight=self.w[1], **kw)

    def check(self, q, out, new, what):
        torch.cuda.synchronize()
        if self.fp8:
            read = [oracle.window.pool_reader(p.cpu().numpy(), s) for p, s in zip((self.pk, self.pv), self.scales)]
        else:
            read = [oracle.window.pool_reader(W.bf16_bits(p)) for p in (self.pk, self.pv)]
        want, terms = oracle.window.extend_attention_window(W.bf16_bits(q), *read, self.rtt, self.rows, self.lens, new,
                                                            self.Hkv, self.window, self.sinks)
        assert_within(W.bf16_bits(out), want, terms, self.fp8, what=what)

    def extend(self, new, **kw):
        q = self.store(new, self.lens, **kw)
        f = B.sgl_extend_attention_window_fp8 if self.fp8 else B.sgl_extend_attention_window
        out = f(q, self.pk, self.pv, *self.scales, self.trtt, self.trows, W.int_tensor(self.lens.astype(np.int32), DEV),
                W.int_tensor(np.array(new, np.int32), DEV), max_extend=max(new), max_prefix=int(self.lens.max()),
                window=self.window, sinks=self.sinks, **kw)
        return q, out

    def decode(self, **kw):
        n = len(self.rows)
        q = self.store([1] * n, self.lens, **kw)
        seq = self.lens + 1
        f = B.sgl_decode_attention_window_fp8 if self.fp8 else B.sgl_decode_attention_window
        out = f(q, self.pk, self.pv, *self.scales, self.trtt, self.trows, W.int_tensor(seq.astype(np.int32), DEV),
                max_seq_len=int(seq.max()), window=self.window, sinks=self.sinks, **kw)
        return q, out


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
def test_a_chunk_then_single_tokens(fp8):
    layer = Layer(1, fp8)
    q, out = layer.extend([50, 9, 33])
    layer.check(q, out, [50, 9, 33], "chunk")
    layer.lens += [50, 9, 33]
    for step in range(4):
        q, out = layer.decode()
        layer.check(q, out, [1, 1, 1], f"token {step}")
        layer.lens += 1


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
def test_on_a_side_stream_with_scratch_of_its_own(fp8):
    """Every buffer the calls make belongs to the stream they run on: nothing
    else may be handed that memory while their kernels run."""
    layer = Layer(2, fp8, prefix=(900, 40, 0), ext=(60, 9, 33), window=500)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(3):
        q, out = layer.extend([60, 9, 33], stream=side)
        # the current stream allocates and overwrites as fast as it can
        for _ in range(20):
            torch.full((1 << 20,), float("nan"), device=DEV)
        layer.check(q, out, [60, 9, 33], "side stream")
    q, out = layer.decode(stream=side.cuda_stream)
    for _ in range(20):
        torch.full((1 << 20,), float("nan"), device=DEV)
    layer.check(q, out, [1, 1, 1], "raw stream handle")


def test_two_calls_at_once_on_two_streams():
    a, b = Layer(3, False, window=64), Layer(4, True, window=300, prefix=(800, 10, 3), ext=(20, 9, 33))
    torch.cuda.synchronize()
    s = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(4):
        qa, oa = a.extend([50, 9, 33], stream=s[0])
        qb, ob = b.extend([20, 9, 33], stream=s[1])
        a.check(qa, oa, [50, 9, 33], "a")
        b.check(qb, ob, [20, 9, 33], "b")


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
def test_captured_and_replayed(fp8):
    """A captured step replays on what its buffers hold then; workspaces may be
    shared by graphs that run one after the other, and by eager calls of other
    sizes between them."""
    cases = [Case(attention_case(40 + i, Hq=8, Hkv=4, D=128, prefix=[700, 3, 90], ext=[1, 1, 1], window=300, sinks=4,
                                 fp8=fp8)) for i in range(2)]
    other = Case(attention_case(50, Hq=4, Hkv=1, D=64, prefix=[2000], ext=[7], window=1500, sinks=2, fp8=fp8))
    dims = B.make_dims(8, 4, 128, cases[0].c["S"])
    od = B.make_dims(4, 1, 64, other.c["S"])
    nbytes = max(B.decode_window_workspace_bytes(3, 701, 300, 4, dims),
                 B.extend_window_workspace_bytes(3, 3, 1, 700, 300, 4, dims),
                 B.extend_window_workspace_bytes(1, 7, 7, 2000, 1500, 2, od))
    ws = B.new_workspace(nbytes, DEV)
    outs = [[torch.empty_like(c.q) for _ in range(2)] for c in cases]
    graphs = []
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        for c, o in zip(cases, outs):
            c.decode(out=o[0], workspace=ws)
            c.extend(out=o[1], workspace=ws)
            side.synchronize()
            graphs.append(torch.cuda.CUDAGraph())
            with torch.cuda.graph(graphs[-1], stream=side):
                c.decode(out=o[0], workspace=ws)
                c.extend(out=o[1], workspace=ws)
    for c, o in zip(cases, outs):
        for t in o:
            t.fill_(float("nan"))
    torch.cuda.synchronize()
    for i in (0, 1, 0, 1):
        graphs[i].replay()
        assert_within(W.bf16_bits(other.extend(workspace=ws)), *other.want_extend(), fp8)
    torch.cuda.synchronize()
    for c, o in zip(cases, outs):
        want, terms = c.want_extend()
        for t in o:
            assert_within(W.bf16_bits(t), want, terms, fp8)
    # new queries in the captured buffers
    cases[0].q.copy_(cases[1].q)
    cases[0].c["q"] = cases[1].c["q"]
    graphs[0].replay()
    torch.cuda.synchronize()
    want, terms = cases[0].want_extend()
    for t in outs[0]:
        assert_within(W.bf16_bits(t), want, terms, fp8)


def test_captured_norm_rope_store():
    c = RopeCase(60, n=33, Hq=8, Hkv=2, D=128)
    out = torch.empty(33, 8, 128, dtype=torch.bfloat16, device=DEV)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        c.run(q_out=out)
        side.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            c.run(q_out=out)
    for p, bits in zip(c.tpool, c.pool):
        p.copy_(W.bf16_tensor(bits, DEV))
    out.zero_()
    torch.cuda.synchronize()
    g.replay()
    torch.cuda.synchronize()
    c.check(out)


def test_what_follows_a_call_of_short_requests_waits_for_it():
    """max_seq_len allows runs, but every request fits one: the combine finds
    nothing to do, and the copy behind it must still see the outputs."""
    case = decode_case(61, [200] * 96, Hq=16, Hkv=8, D=128, window=4096, sinks=4)
    want, terms = case.want_decode()
    for _ in range(10):
        out = torch.full_like(case.q, float("nan"))
        case.decode(out=out, max_seq_len=32768)
        got = out.clone()
        assert_within(W.bf16_bits(got), want, terms, False)


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("dealt", [True, False])
def test_extend_gives_up_then_recovers(dealt, fp8):
    shape = dict(Hq=4, Hkv=2, D=128, prefix=[900, 30], ext=[60, 9]) if dealt else \
        dict(Hq=64, Hkv=64, D=64, prefix=[300, 30, 7], ext=[60, 9, 2])
    case = Case(attention_case(62, window=700, sinks=4, fp8=fp8, **shape))
    c = case.c
    nbytes = B.extend_window_workspace_bytes(len(c["ext"]), int(c["ext"].sum()), 60, int(c["prefix"].max()), 700, 4,
                                             B.make_dims(c["Hq"], c["Hkv"], c["D"], c["S"]))
    assert (nbytes > 256) == dealt
    ws = B.new_workspace(nbytes, DEV)
    with short_waits():
        case.extend(workspace=ws)
    assert int(ws[:4].view(torch.int32).item()) == TIMEOUT_CODE
    ws = B.new_workspace(nbytes, DEV)
    assert_within(W.bf16_bits(case.extend(workspace=ws)), *case.want_extend(), fp8)
    assert int(ws[:4].view(torch.int32).item()) == 0


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
def test_slots_past_32_bit_offsets(fp8):
    """Pools of more than 2^32 bytes and 2^31 values, the slots at their end."""
    small = attention_case(63, Hq=8, Hkv=8, D=128, prefix=[400, 3], ext=[5, 1], window=200, sinks=4, fp8=fp8)
    S, n = ((1 << 32) // 1024 if fp8 else (1 << 31) // 1024) + 4096, small["S"]
    big = dict(small, S=S, rtt=small["rtt"] + np.int32(S - n))
    case = Case(dict(small))
    for name in ("pk", "pv"):
        pool = torch.empty((S,) + tuple(getattr(case, name).shape[1:]), dtype=getattr(case, name).dtype, device=DEV)
        pool[S - n:] = getattr(case, name)
        setattr(case, name, pool)
    case.rtt = W.int_tensor(big["rtt"], DEV)
    want, terms = case.want_extend()
    assert_within(W.bf16_bits(case.extend()), want, terms, fp8, what="extend")
    # the same requests' last tokens as decodes
    rows = [4, 5]
    q = case.q
    case.q = q[rows].contiguous()
    assert_within(W.bf16_bits(case.decode()), want[rows], {k: v[rows] for k, v in terms.items()}, fp8, what="decode")
    # rows stored there
    x = q[:, :8].contiguous()
    slots = torch.arange(S - 6, S, dtype=torch.int32, device=DEV)
    if fp8:
        B.sgl_qk_norm_rope_store_kv_fp8(x, x, x, None, None, slots, case.pk, case.pv, 0.25, 0.25)
        near = torch.zeros(8, 8, 128, dtype=torch.uint8, device=DEV), torch.zeros(8, 8, 128, dtype=torch.uint8, device=DEV)
        B.sgl_store_kv_fp8(x, x, torch.arange(6, dtype=torch.int32, device=DEV), *near, 0.25, 0.25)
        assert torch.equal(case.pk[S - 6:], near[0][:6]) and torch.equal(case.pv[S - 6:], near[1][:6])
    else:
        B.sgl_qk_norm_rope_store_kv(x, x, x, None, None, slots, case.pk, case.pv)
        assert torch.equal(case.pk[S - 6:], x) and torch.equal(case.pv[S - 6:], x)


def test_shared_rows_and_the_same_request_twice():
    """Two requests may name the same row of req_to_token."""
    case = decode_case(64, [300, 300], Hq=8, Hkv=2, D=64, window=90, sinks=2)
    case.c["rpi"] = case.c["rpi"][[0, 0]]
    case.rpi = W.int_tensor(case.c["rpi"], DEV)
    check_decode(case, case.decode())


def test_queries_may_be_overwritten_by_the_output():
    case = Case(attention_case(65, Hq=8, Hkv=2, D=64, prefix=[100, 3], ext=[40, 9], window=30, sinks=2))
    want = case.want_extend()
    case.extend(out=case.q)
    assert_within(W.bf16_bits(case.q), *want, False)
    for seq, window in (([300, 7], 40), ([3000, 900], 2500)):
        case = decode_case(66, seq, Hq=8, Hkv=2, D=64, window=window, sinks=2)
        want = case.want_decode()
        case.decode(out=case.q)
        assert_within(W.bf16_bits(case.q), *want, False)
