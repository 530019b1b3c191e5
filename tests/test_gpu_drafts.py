"""Drafted tokens on the GPU against the fp64 oracle: attention within the bounds
derived in _drafts.py (hidden positions' entries of req_to_token point at NaN rows),
kept nodes, drawn tokens and slots exactly."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import oracle  # noqa: E402
from radixattention_prefix_shared_gb300 import binding as B  # noqa: E402
from radixattention_prefix_shared_gb300 import workloads as W  # noqa: E402

from _drafts import accept_case, assert_attention, attention_case, tree, want_accept  # noqa: E402
from test_gpu_wait_timeout import TIMEOUT_CODE, short_waits  # noqa: E402

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]

DEV = "cuda:0"


class Case:
    """An attention case's inputs on the GPU and the call over them."""

    def __init__(self, c):
        self.c = c
        self.q = W.bf16_tensor(c["q"], DEV)
        up = (lambda x: torch.from_numpy(x).to(DEV)) if c["fp8"] else (lambda x: W.bf16_tensor(x, DEV))
        self.pk, self.pv = up(c["pool_k"]), up(c["pool_v"])
        self.rtt, self.rpi, self.prefix, self.drafts, self.parents = (
            W.int_tensor(c[n], DEV) for n in ("rtt", "rpi", "prefix", "drafts", "parents"))
        self.scales = (c["k_scale"], c["v_scale"]) if c["fp8"] else ()

    def maxima(self):
        c = self.c
        return dict(max_draft=max(1, int(c["drafts"].max())), max_prefix=int(c["prefix"].max()),
                    shared_len=c["shared"])

    def new_workspace(self, **kw):
        c, a = self.c, self.maxima() | kw
        return B.new_workspace(B.verify_workspace_bytes(len(c["rpi"]), len(c["parents"]), a["max_draft"],
                                                        a["max_prefix"], a["shared_len"],
                                                        B.make_dims(c["Hq"], c["Hkv"], c["D"], c["S"])), DEV)

    def run(self, **kw):
        f = B.sgl_verify_attention_fp8 if self.c["fp8"] else B.sgl_verify_attention
        return f(self.q, self.pk, self.pv, *self.scales, self.rtt, self.rpi, self.prefix, self.drafts, self.parents,
                 **(self.maxima() | kw))

    def check(self, what="", **kw):
        ws = self.new_workspace()
        out = self.run(workspace=ws, **kw)
        assert int(ws[:4].view(torch.int32).item()) == 0, "a wait gave up"
        assert_attention(W.bf16_bits(out), self.c, what)
        return out


SHAPES = [(4, 4, 64), (4, 4, 128), (6, 2, 128), (8, 2, 64), (16, 2, 128), (5, 1, 64), (24, 3, 128)]


# ------------------------------------------------------------------ attention

@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("Hq,Hkv,D", SHAPES)
@pytest.mark.parametrize("kind", ["tree", "chain", "bush", "forest"])
def test_small(Hq, Hkv, D, kind, fp8):
    """Prefixes that end in every part of a 128-key block, trees across its edge."""
    Case(attention_case(10, Hq=Hq, Hkv=Hkv, D=D, prefix=[0, 1, 120, 127, 128, 129, 250, 383],
                        drafts=[1, 5, 16, 2, 7, 9, 12, 3], kind=kind, fp8=fp8)).check()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("n", [1, 2, 4, 8, 16, 33, 63, 64])
def test_tile_widths(n, fp8):
    """Every width of a tile, full and partly so, and several tiles a request."""
    for Hq, Hkv in ((2, 2), (4, 1), (7, 1)):
        Case(attention_case(11 + n, Hq=Hq, Hkv=Hkv, D=128, prefix=[300, 65, 0], drafts=[n, max(1, n - 1), n],
                            fp8=fp8)).check(f"{n} nodes, {Hq} on {Hkv}")


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("D", [64, 128])
def test_a_head_group_wider_than_a_tile(D, fp8):
    Case(attention_case(13, Hq=128, Hkv=1, D=D, prefix=[140, 3], drafts=[3, 2], fp8=fp8)).check()
    Case(attention_case(14, Hq=200, Hkv=2, D=D, prefix=[140, 3], drafts=[3, 2], fp8=fp8)).check()


@pytest.mark.parametrize("fp8", [False, True])
def test_long_prefixes_are_split_and_joined(fp8):
    """One request's keys over most CTAs; CTAs that hold parts of several units."""
    Case(attention_case(15, Hq=8, Hkv=2, D=128, prefix=[20011], drafts=[5], fp8=fp8)).check("one long")
    Case(attention_case(16, Hq=4, Hkv=1, D=64, prefix=[5000, 1, 0, 7777, 300], drafts=[9, 1, 64, 2, 17],
                        fp8=fp8)).check("ragged")


@pytest.mark.parametrize("fp8", [False, True])
def test_many_requests(fp8):
    """More requests than a warp lists at a time, many of them padding."""
    g = np.random.default_rng(17)
    n = [int(x) for x in g.choice([0, 0, 0, 1, 2, 5], size=300)]
    Case(attention_case(17, Hq=4, Hkv=2, D=64, prefix=[int(x) for x in g.integers(0, 200, size=300)], drafts=n,
                        fp8=fp8)).check()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("shared", [1, 127, 128, 129, 700])
def test_a_shared_prefix_is_read_once(shared, fp8):
    c = attention_case(18 + shared, Hq=8, Hkv=2, D=128, prefix=[700, 701, 900, 700, 1500], drafts=[4, 0, 9, 1, 20],
                       shared=shared, fp8=fp8)
    case = Case(c)
    one = case.check()
    # the rows' own shared entries are not looked at, but for the first request's
    first = int(c["rpi"][0])
    other = c["rtt"].copy()
    other[[r for r in range(other.shape[0]) if r != first], :shared] = c["rtt"][(first + 1) % 3, -1]
    case.rtt = W.int_tensor(other, DEV)
    assert torch.equal(one.view(torch.int16), case.run().view(torch.int16))


def test_shared_prefix_of_many_rows():
    """The batch's rows fill many tiles."""
    Case(attention_case(19, Hq=8, Hkv=2, D=128, prefix=[520] * 40, drafts=[8] * 40, shared=512)).check()
    Case(attention_case(20, Hq=8, Hkv=2, D=64, prefix=[520] * 30, drafts=[7] * 30, shared=300, fp8=True)).check()


@pytest.mark.parametrize("fp8", [False, True])
def test_references_move(fp8):
    """Scores that grow by hundreds along the keys: references move many times, and a
    first block far below the rest leaves nothing behind."""
    c = attention_case(21, Hq=2, Hkv=1, D=64, prefix=[1500], drafts=[6], std=1.0)
    g = np.random.default_rng(21)
    grow = np.linspace(-12, 12, 1506)
    k = g.standard_normal((c["S"], 1, 64)).astype(np.float32) * 0.1
    slots = c["rtt"][c["rpi"][0], :1506]
    q = np.abs(g.standard_normal((6, 2, 64)).astype(np.float32)) + 0.5
    k[slots] += grow[:, None, None].astype(np.float32)
    c["q"], c["pool_k"] = W.f32_to_bf16_bits(q), W.f32_to_bf16_bits(k)
    if fp8:
        c["fp8"], c["k_scale"], c["v_scale"] = True, 0.05, 0.0173
        c["pool_k"] = oracle.fp8.quantize(c["pool_k"], 0.05)
        live = np.zeros(c["S"], bool)
        live[slots] = True
        v = np.where(live[:, None, None], c["pool_v"], 0)
        c["pool_v"] = oracle.fp8.quantize(v.astype(np.uint16), 0.0173)
    Case(c).check()


@pytest.mark.parametrize("fp8", [False, True])
def test_rows_behind_the_last_node_stay(fp8):
    c = attention_case(22, Hq=4, Hkv=2, D=64, prefix=[30, 400], drafts=[3, 2], fp8=fp8)
    pad = 9
    c["q"] = np.concatenate([c["q"], np.full((pad,) + c["q"].shape[1:], 0x7FC0, np.uint16)])
    c["parents"] = np.concatenate([c["parents"], np.full(pad, 99, np.int32)])
    case = Case(c)
    out = torch.full_like(case.q, 3.0)
    case.check(out=out)
    assert (out[5:] == 3.0).all()


def test_output_over_the_queries():
    case = Case(attention_case(23, Hq=8, Hkv=2, D=128, prefix=[3000, 5, 700], drafts=[4, 9, 1]))
    want = case.run()
    got = case.run(out=case.q)
    assert got.data_ptr() == case.q.data_ptr() and torch.equal(got.view(torch.int16), want.view(torch.int16))


def test_maxima_above_the_lengths():
    """Host maxima are bounds: what they are above the lengths changes no key."""
    c = attention_case(24, Hq=4, Hkv=2, D=128, prefix=[30, 400], drafts=[3, 7])
    case = Case(c)
    ws = case.new_workspace(max_draft=10, max_prefix=401)
    assert_attention(W.bf16_bits(case.run(max_draft=10, max_prefix=401, workspace=ws)), c)


@pytest.mark.parametrize("fp8", [False, True])
def test_scale_of_the_callers_choice(fp8):
    c = attention_case(28, Hq=4, Hkv=2, D=128, prefix=[70, 700], drafts=[6, 3], fp8=fp8)
    case = Case(c)
    out = W.bf16_bits(case.run(sm_scale=0.031))
    want, _ = oracle.drafts.verify_attention(
        c["q"], *(oracle.window.pool_reader(c["pool_" + x], c[x + "_scale"]) for x in "kv"), c["rtt"], c["rpi"],
        c["prefix"], c["drafts"], c["parents"], 2, sm_scale=0.031)
    # as in _drafts.py, with sum p |V| <= max |V|; scores here are below 2^4
    bound = 2.0 ** -8 * np.abs(want) + (2.0 ** -8 + 2.0 ** -12 + 2.0 ** -12) * 6 * (1 if not fp8 else 2)
    assert (np.abs(oracle.bf16_bits_to_f64(out) - want) <= bound).all()
    # (another scale is another result)
    assert np.abs(oracle.bf16_bits_to_f64(out) - oracle.bf16_bits_to_f64(W.bf16_bits(case.run()))).max() > 0.05


def test_a_batch_of_padding_and_rows_that_end_with_their_nodes():
    """No request has nodes: nothing is written.  A prefix and its nodes that fill a
    row of the table to its end."""
    c = attention_case(29, Hq=4, Hkv=2, D=64, prefix=[5, 60], drafts=[0, 0])
    case = Case(c)
    for shared in (0, 5):
        out = torch.full_like(case.q, 2.0)
        case.run(out=out, max_draft=1, shared_len=shared)
        assert (out == 2.0).all()
    c = attention_case(30, Hq=4, Hkv=2, D=64, prefix=[130, 60], drafts=[7, 9])
    c["rtt"] = np.ascontiguousarray(c["rtt"][:, :137])
    Case(c).check(max_prefix=130)


def test_fewer_tokens_than_rows():
    c = attention_case(31, Hq=4, Hkv=2, D=64, prefix=[30, 200], drafts=[3, 4])
    c["q"] = np.concatenate([c["q"], c["q"][:2]])
    c["parents"] = np.concatenate([c["parents"], c["parents"][:2]])
    case = Case(c)
    out = torch.full_like(case.q, 2.0)
    case.check(out=out, total_draft=7)
    assert (out[7:] == 2.0).all()


def test_parents_that_are_none():
    """A parent outside [0, node) is none: the node sees the prefix and itself."""
    c = attention_case(25, Hq=2, Hkv=1, D=64, prefix=[50], drafts=[6])
    c["parents"] = np.array([5, 1, 0, 3, 2, 2**31 - 1], np.int32)
    Case(c).check()


def test_offsets_past_32_bits():
    """Slots whose bytes lie past 2^32 in the pools."""
    S, Hkv, D = 2**32 // (8 * 128 * 2) + 4096, 8, 128
    g = np.random.default_rng(26)
    pk = torch.zeros(S, Hkv, D, dtype=torch.bfloat16, device=DEV)
    pv = torch.zeros_like(pk)
    n, p = 4, 300
    slots = (S - 1 - g.permutation(p + n)).astype(np.int32)
    k, v = (W.f32_to_bf16_bits(g.standard_normal((p + n, Hkv, D)).astype(np.float32)) for _ in range(2))
    at = torch.from_numpy(slots.astype(np.int64)).to(DEV)
    pk[at], pv[at] = W.bf16_tensor(k, DEV), W.bf16_tensor(v, DEV)
    c = dict(Hq=8, Hkv=Hkv, D=D, S=p + n, shared=0, rtt=np.arange(p + n, dtype=np.int32)[None], rpi=np.zeros(1, np.int32),
             prefix=np.array([p], np.int32), drafts=np.array([n], np.int32), parents=np.array([-1, 0, 0, 2], np.int32),
             fp8=False, k_scale=None, v_scale=None, pool_k=k, pool_v=v,
             q=W.f32_to_bf16_bits(g.standard_normal((n, 8, D)).astype(np.float32)))
    out = B.sgl_verify_attention(W.bf16_tensor(c["q"], DEV), pk, pv, W.int_tensor(slots[None], DEV),
                                 W.int_tensor(c["rpi"], DEV), W.int_tensor(c["prefix"], DEV),
                                 W.int_tensor(c["drafts"], DEV), W.int_tensor(c["parents"], DEV), max_draft=n,
                                 max_prefix=p)
    assert_attention(W.bf16_bits(out), c)


@pytest.mark.parametrize("fp8", [False, True])
def test_waits_give_up_then_recover(fp8):
    case = Case(attention_case(27, Hq=8, Hkv=2, D=128, prefix=[900, 30], drafts=[9, 4], shared=20, fp8=fp8))
    ws = case.new_workspace()
    with short_waits():
        case.run(workspace=ws)
    torch.cuda.synchronize()
    assert int(ws[:4].view(torch.int32).item()) == TIMEOUT_CODE
    case.check("after a call that gave up")


def test_graph_with_new_lengths():
    """A captured step replays with other lengths, trees and table rows than it was
    captured with; two graphs share a workspace in turn."""
    Hq, Hkv, D, b, most, cap = 8, 2, 64, 4, 9, 600
    cs = [attention_case(30 + i, Hq=Hq, Hkv=Hkv, D=D, prefix=p, drafts=n, kind="forest")
          for i, (p, n) in enumerate([([5, 100, 599, 0], [9, 1, 2, 4]), ([300, 2, 1, 600], [1, 9, 9, 0]),
                                      ([0, 0, 0, 0], [1, 1, 1, 1])])]
    T, rows, stride = b * most, 7, cap + most
    S = max(c["S"] for c in cs)
    st = dict(q=torch.zeros(T, Hq, D, dtype=torch.bfloat16, device=DEV),
              pk=torch.zeros(S, Hkv, D, dtype=torch.bfloat16, device=DEV),
              rtt=torch.zeros(rows, stride, dtype=torch.int32, device=DEV),
              parents=torch.zeros(T, dtype=torch.int32, device=DEV))
    st["pv"], st["out"] = torch.zeros_like(st["pk"]), torch.zeros_like(st["q"])
    for n in ("rpi", "prefix", "drafts"):
        st[n] = torch.zeros(b, dtype=torch.int32, device=DEV)
    ws = B.new_workspace(B.verify_workspace_bytes(b, T, most, cap, 0, B.make_dims(Hq, Hkv, D, S)), DEV)

    def fill(c):
        for name, key in (("q", "q"), ("pk", "pool_k"), ("pv", "pool_v")):
            st[name][: len(c[key])].copy_(W.bf16_tensor(c[key], DEV))
        st["rtt"].zero_()
        st["rtt"][: c["rtt"].shape[0], : c["rtt"].shape[1]].copy_(W.int_tensor(c["rtt"], DEV))
        st["parents"][: len(c["parents"])].copy_(W.int_tensor(c["parents"], DEV))
        for n in ("rpi", "prefix", "drafts"):
            st[n].copy_(W.int_tensor(c[n], DEV))

    def step():
        B.sgl_verify_attention(st["q"], st["pk"], st["pv"], st["rtt"], st["rpi"], st["prefix"], st["drafts"],
                               st["parents"], st["out"], max_draft=most, max_prefix=cap, workspace=ws)

    fill(cs[0])
    step()
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            step()
    for i in (1, 0, 2, 1):
        fill(cs[i])
        for graph in graphs:
            st["out"].fill_(7.0)
            graph.replay()
            torch.cuda.synchronize()
            assert_attention(W.bf16_bits(st["out"]), cs[i], f"replay {i}")
    assert int(ws[:4].view(torch.int32).item()) == 0


def test_on_another_stream():
    """Two calls at once, each on its own stream with its own workspace; inputs and
    what the calls allocate may be dropped on return."""
    cs = [attention_case(40 + i, Hq=8, Hkv=2, D=128, prefix=[4000, 90, 2000], drafts=[8, 3, 30], fp8=bool(i))
          for i in range(2)]
    cases = [Case(c) for c in cs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cs]
    outs = [[x.run(stream=s) for _ in range(3)] for x, s in zip(cases, streams)]
    del cases
    junk = [torch.full((1 << 20,), 9.0, device=DEV) for _ in range(40)]
    for s in streams:
        s.synchronize()
    del junk
    for c, o in zip(cs, outs):
        for x in o:
            assert_attention(W.bf16_bits(x), c)


def test_refusals():
    case = Case(attention_case(50, Hq=4, Hkv=2, D=64, prefix=[9, 30], drafts=[2, 3]))
    f = B.sgl_verify_attention
    args = [case.q, case.pk, case.pv, case.rtt, case.rpi, case.prefix, case.drafts, case.parents]
    kw = case.maxima()
    for i, bad in [(0, case.q.float()), (0, case.q[:, :, ::2]), (0, case.q[0]), (0, case.q.cpu()),
                   (1, case.pk.float()), (2, case.pv[1:]), (3, case.rtt.long()), (3, case.rtt[:, ::2]), (4, case.rpi[:1]),
                   (5, case.prefix[:1]), (6, case.drafts.float()), (7, case.parents[:-1])]:
        with pytest.raises(ValueError):
            f(*[bad if j == i else a for j, a in enumerate(args)], **kw)
    with pytest.raises(ValueError):
        f(*args, out=case.q[:-1], **kw)
    for name in ("max_draft", "max_prefix", "shared_len"):
        for bad in (2**31, 2**40, -2**31):
            with pytest.raises(ValueError, match=name):
                f(*args, **(kw | {name: bad}))
    with pytest.raises(ValueError, match="total_draft"):
        f(*args, total_draft=6, **kw)
    with pytest.raises(B.SglError) as e:
        f(*args, workspace=B.new_workspace(64, DEV), **kw)
    assert e.value.code == 3
    with pytest.raises(B.SglError) as e:
        f(*args, **(kw | dict(max_prefix=case.rtt.shape[1])))
    assert e.value.code == 1


def _checked(case, **kw):
    err = torch.zeros(4, dtype=torch.int32, device=DEV)
    a = dict(total_draft=int(np.maximum(case.c["drafts"], 0).sum()), pool_size=case.c["S"], d_error=err, **case.maxima())
    B.sgl_check_verify_indices(case.rtt, case.rpi, case.prefix, case.drafts, case.parents, **(a | kw))
    return err.tolist()


def test_checked_mode():
    new = lambda: attention_case(51, Hq=4, Hkv=2, D=64, prefix=[40, 3, 50], drafts=[4, 0, 3], shared=30)  # noqa: E731
    assert _checked(Case(new())) == [0, 0, 0, 0]
    bad = new()
    bad["rtt"][bad["rpi"][2], 51] = bad["S"]
    assert _checked(Case(bad))[:3] == [1, 2, 51]
    bad = new()
    bad["rpi"][0] = 77
    assert _checked(Case(bad))[:2] == [2, 0]
    bad = new()
    bad["prefix"][2] = -1
    assert _checked(Case(bad), max_prefix=40)[0] == 3
    assert _checked(Case(new()), total_draft=8)[0] == 5 and _checked(Case(new()), max_draft=3)[0] == 5
    bad = new()
    bad["parents"][6] = 2
    assert _checked(Case(bad)) == [11, 2, 2, 2]
    bad = new()
    bad["rtt"][bad["rpi"][2], 7] = bad["rtt"][bad["rpi"][2], 40]
    assert _checked(Case(bad))[:3] == [12, 2, 7]
    assert _checked(Case(new()), shared_len=45)[0] == 12


# ------------------------------------------------------------------ the walk

def run_accept(c, p=None, q=None, **kw):
    up = lambda x: torch.from_numpy(x).to(DEV)  # noqa: E731
    p = up(c["p"]) if p is None else p
    q = (up(c["q"]) if c["q"] is not None else None) if q is None else q
    out = B.sgl_verify_drafts(p, up(c["tok"]), up(c["parents"]), up(c["drafts"]), up(c["coins"]), up(c["final"]), q,
                              **(dict(max_draft=c["most"]) | kw))
    return [x.cpu().numpy() for x in out]


def check_accept(c, **kw):
    for name, got, want in zip(("accepted", "num_accepted", "next_tokens"), run_accept(c, **kw), want_accept(c)):
        assert np.array_equal(got, want), (name, got, want)


@pytest.mark.parametrize("drawn", [True, False])
@pytest.mark.parametrize("V", [1, 2, 3, 31, 128, 1000, 4097, 50257])
@pytest.mark.parametrize("kind", ["chain", "tree", "bush"])
def test_walks(V, kind, drawn):
    check_accept(accept_case(60 + V, drafts=[1, 5, 0, 2, 12, 7, 0, 3], V=V, kind=kind, drawn=drawn))


@pytest.mark.parametrize("drawn", [True, False])
def test_full_trees_and_large_batches(drawn):
    check_accept(accept_case(70, drafts=[64, 63, 1, 64], V=5000, drawn=drawn))
    check_accept(accept_case(71, drafts=[64, 33], V=700, kind="bush", drawn=drawn))
    g = np.random.default_rng(72)
    check_accept(accept_case(72, drafts=[int(x) for x in g.integers(0, 4, size=400)], V=900, drawn=drawn))
    # one CTA a request, several parts a warp
    check_accept(accept_case(73, drafts=[1] * 470, V=20011, drawn=drawn))
    check_accept(accept_case(74, drafts=[3, 2], V=300001, drawn=drawn))


@pytest.mark.parametrize("drawn", [True, False])
def test_rows_apart_and_out_of_step(drawn):
    """Rows of padded vocabularies; a draft tensor that lies otherwise against 16 bytes."""
    c = accept_case(75, drafts=[6, 1, 9, 4], V=5003, drawn=drawn)
    want = want_accept(c)
    T = len(c["tok"])
    for ld, at, qld, qat in ((5003, 0, 5003, 0), (5120, 1, 5120, 1), (5010, 3, 5007, 2), (5004, 0, 5005, 1)):
        p = torch.full((T, ld + 8), float("nan"), device=DEV)
        p[:, at: at + 5003] = torch.from_numpy(c["p"]).to(DEV)
        q = None
        if drawn:
            q = torch.full((T, qld + 8), float("nan"), device=DEV)
            q[:, qat: qat + 5003] = torch.from_numpy(c["q"]).to(DEV)
            q = q[:, qat: qat + 5003]
        for got, w in zip(run_accept(c, p=p[:, at: at + 5003], q=q), want):
            assert np.array_equal(got, w)


def test_walk_corner_cases():
    c = accept_case(76, drafts=[4, 3, 2, 1, 5], V=40, drawn=False, kind="bush")
    c["tok"][[1, 2, 3]] = [7, 7, 7]            # the same token among siblings
    c["tok"][[5, 6]] = [-1, 40]                # outside the vocabulary
    c["coins"][[1, 2]] = 1.0
    c["p"][7] = 0.0                            # a row without weights
    c["p"][9] = [np.nan, -1.0, np.inf] + [0.0] * 36 + [0.25]
    c["final"][:] = [0.0, np.float32(1 - 2**-24), 0.5, 0.5, 0.0]
    c["parents"][12] = 9                       # a parent behind its node
    check_accept(c)
    got = run_accept(c)
    assert got[2][2] == -1 and got[2][3] == 39
    # nothing is left of R: the target row itself
    c = accept_case(77, drafts=[2], V=10, drawn=True)
    c["q"] = c["p"].copy()
    c["coins"][:] = 1.0
    check_accept(c)
    # a coin of 1: the last weight's token
    c = accept_case(78, drafts=[1, 1], V=3000, drawn=True)
    c["p"][:, 2900:] = 0.0
    c["final"][:] = 1.0
    assert run_accept(c)[2].tolist() == [2899, 2899]


def test_walk_outputs_given_and_captured():
    c = accept_case(79, drafts=[5, 0, 3], V=2000, drawn=True)
    up = lambda x: torch.from_numpy(x).to(DEV)  # noqa: E731
    args = [up(c[k]) for k in ("p", "tok", "parents", "drafts", "coins", "final", "q")]
    out = dict(accepted=torch.empty(3, 8, dtype=torch.int32, device=DEV),
               num_accepted=torch.empty(3, dtype=torch.int32, device=DEV),
               next_tokens=torch.empty(3, dtype=torch.int32, device=DEV))
    B.sgl_verify_drafts(*args, max_draft=8, **out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.sgl_verify_drafts(*args, max_draft=8, **out)
    c2 = accept_case(80, drafts=[1, 5, 2], V=2000, drawn=True)
    for a, k in zip(args, ("p", "tok", "parents", "drafts", "coins", "final", "q")):
        a.copy_(up(c2[k]))
    graph.replay()
    torch.cuda.synchronize()
    want = want_accept(c2 | dict(most=8))
    for k, w in zip(("accepted", "num_accepted", "next_tokens"), want):
        assert np.array_equal(out[k].cpu().numpy(), w), k
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = B.sgl_verify_drafts(*args, max_draft=8, stream=s)
    del args
    s.synchronize()
    assert np.array_equal(got[0].cpu().numpy(), want[0])


def test_walk_refusals():
    c = accept_case(81, drafts=[3, 2], V=50, drawn=True)
    up = lambda x: torch.from_numpy(x).to(DEV)  # noqa: E731
    args = [up(c[k]) for k in ("p", "tok", "parents", "drafts", "coins", "final", "q")]
    for i, bad in [(0, args[0].double()), (0, args[0].t()), (0, args[0].cpu()), (1, args[1].long()), (1, args[1][:-1]),
                   (2, args[2][:-1]), (3, args[3].float()), (4, args[4].double()), (5, args[5][:1]), (6, args[6][:, :-1])]:
        with pytest.raises(ValueError):
            B.sgl_verify_drafts(*[bad if j == i else a for j, a in enumerate(args)], max_draft=3)
    for bad in (0, 65, -1):
        with pytest.raises(ValueError, match="max_draft"):
            B.sgl_verify_drafts(*args, max_draft=bad)
    with pytest.raises(ValueError):
        B.sgl_verify_drafts(*args, max_draft=3, accepted=torch.empty(2, 4, dtype=torch.int32, device=DEV))


# ------------------------------------------------------------------ slots

def commit_case(seed, drafts, *, most=None, kind="tree", stride=900):
    g = np.random.default_rng(seed)
    n = [max(0, x) for x in drafts]
    T, b, most = max(1, sum(n)), len(n), most or max(1, max(n, default=1))
    acc, cnt = np.full((b, most), -1, np.int32), np.zeros(b, np.int32)
    for r, x in enumerate(n):
        if x:
            line = oracle.drafts.line_of(tree(g, x, kind), int(g.integers(0, x)))
            acc[r, : len(line)], cnt[r] = line, len(line)
    return dict(rtt=g.integers(0, 99, size=(b + 2, stride)).astype(np.int32), rpi=g.permutation(b + 2)[:b].astype(np.int32),
                pre=g.integers(0, stride - 64, size=b).astype(np.int32), drafts=np.asarray(drafts, np.int32),
                slots=(1000 + g.permutation(T)).astype(np.int32), acc=acc, cnt=cnt)


def run_commit(c, **kw):
    t = {k: torch.from_numpy(v).to(DEV) for k, v in c.items()}
    out = B.sgl_commit_drafts(t["rtt"], t["rpi"], t["pre"], t["drafts"], t["slots"], t["acc"], t["cnt"], **kw)
    return t["rtt"].cpu().numpy(), *[x.cpu().numpy() for x in out]


@pytest.mark.parametrize("drafts", [[1], [5], [64], [0], [3, 0, 64, 1, 17, 0, 2], [7] * 200, [0] * 5 + [9]])
def test_commit(drafts):
    c = commit_case(90, drafts)
    table, seq, freed, count = run_commit(c, freed=torch.full((len(c["slots"]),), -5, dtype=torch.int32, device=DEV))
    want = oracle.drafts.commit_drafts(c["rtt"], c["rpi"], c["pre"], c["drafts"], c["slots"], c["acc"], c["cnt"])
    assert np.array_equal(table, want[0]) and np.array_equal(seq, want[1])
    assert count.tolist() == [len(want[2])] and np.array_equal(freed[: len(want[2])], want[2])
    assert (freed[len(want[2]):] == -5).all()


def test_commit_skips_what_it_cannot_place():
    c = commit_case(91, [4, 4], stride=80)
    c["acc"][:] = [[0, 1, 9, -3], [0, 2, -1, -1]]
    c["cnt"][:] = [4, 2]
    c["pre"][:] = [10, 79]      # the second path's last position lies behind its row
    table, seq, freed, count = run_commit(c)
    want = c["rtt"].copy()
    want[c["rpi"][0], 10:12] = c["slots"][:2]
    want[c["rpi"][1], 79] = c["slots"][4]
    assert np.array_equal(table, want) and seq.tolist() == [14, 81]
    assert count.tolist() == [2] and freed[:2].tolist() == c["slots"][[5, 7]].tolist()
    c["rpi"][:] = [-1, 99]
    assert np.array_equal(run_commit(c)[0], c["rtt"])


def test_commit_refusals():
    c = commit_case(92, [3, 2])
    t = {k: torch.from_numpy(v).to(DEV) for k, v in c.items()}
    for k, bad in [("rtt", t["rtt"].long()), ("rtt", t["rtt"][0]), ("rpi", t["rpi"][:1]), ("pre", t["pre"].float()),
                   ("drafts", t["drafts"].cpu()), ("acc", t["acc"][:1]), ("cnt", t["cnt"][:1]), ("slots", t["slots"][None])]:
        a = t | {k: bad}
        with pytest.raises(ValueError):
            B.sgl_commit_drafts(a["rtt"], a["rpi"], a["pre"], a["drafts"], a["slots"], a["acc"], a["cnt"])
    with pytest.raises(ValueError, match="max_draft"):
        B.sgl_commit_drafts(t["rtt"], t["rpi"], t["pre"], t["drafts"], t["slots"],
                            torch.zeros(2, 65, dtype=torch.int32, device=DEV), t["cnt"])
    empty = torch.zeros(0, dtype=torch.int32, device=DEV)
    out = B.sgl_commit_drafts(t["rtt"], empty, empty, empty, empty, torch.zeros(0, 3, dtype=torch.int32, device=DEV), empty)
    assert out[2].tolist() == [0]


# ------------------------------------------------------------------ a whole step

@pytest.mark.parametrize("fp8", [False, True])
def test_steps_of_a_loop(fp8):
    """Three steps: the drafted tokens' K and V are stored by the norm + rotation +
    store call (at prefix + depth), attended to, walked, and the kept ones committed;
    then a decode over the committed rows equals one over rows that held those tokens
    alone."""
    g = np.random.default_rng(95)
    Hq, Hkv, D, V, b, most, cap = 8, 2, 64, 500, 3, 7, 200
    S = 2000
    scales = (0.05, 0.03) if fp8 else ()
    pool = [torch.zeros(S, Hkv, D, dtype=torch.uint8 if fp8 else torch.bfloat16, device=DEV) for _ in range(2)]
    free = list(g.permutation(S).astype(int))
    rtt = torch.full((b, cap), -1, dtype=torch.int32, device=DEV)
    rows = torch.arange(b, dtype=torch.int32, device=DEV)
    f = torch.from_numpy((1e4 ** (-np.arange(0, D, 2) / D)).astype(np.float32)).to(DEV)
    tail = "_fp8" if fp8 else ""
    lens = np.array([20, 1, 130], np.int32)
    kept_rows = [[] for _ in range(b)]

    def store(positions, slots, n):
        x = W.bf16_tensor(W.f32_to_bf16_bits(g.standard_normal((n, Hq + 2 * Hkv, D)).astype(np.float32)), DEV)
        q, k, v = x.split([Hq, Hkv, Hkv], dim=1)
        return getattr(B, "sgl_qk_norm_rope_store_kv" + tail)(
            q, k, v, W.int_tensor(np.asarray(positions, np.int32), DEV), f, W.int_tensor(np.asarray(slots, np.int32), DEV),
            *pool, *scales)

    for r, n in enumerate(lens):
        slots = [free.pop() for _ in range(n)]
        store(range(n), slots, int(n))
        rtt[r, :n] = torch.tensor(slots, dtype=torch.int32, device=DEV)
        kept_rows[r] = slots
    for step in range(3):
        n = [int(x) for x in g.integers(1, most + 1, size=b)]
        par = [tree(g, x, "tree") for x in n]
        flat = np.asarray([v for p in par for v in p], np.int32)
        slots = np.asarray([free.pop() for _ in range(sum(n))], np.int32)
        depth = [len(oracle.drafts.line_of(p, i)) - 1 for p in par for i in range(len(p))]
        start = np.repeat(lens, n)
        q = store(start + np.asarray(depth), slots, sum(n))
        at = 0
        for r in range(b):
            rtt[r, lens[r]: lens[r] + n[r]] = W.int_tensor(slots[at: at + n[r]], DEV)
            at += n[r]
        pre, dl, parents = (W.int_tensor(np.asarray(x, np.int32), DEV) for x in (lens, n, flat))
        out = getattr(B, "sgl_verify_attention" + tail)(q, *pool, *scales, rtt, rows, pre, dl, parents, max_draft=most,
                                                        max_prefix=cap - most)
        c = dict(Hq=Hq, Hkv=Hkv, D=D, rtt=rtt.cpu().numpy(), rpi=rows.cpu().numpy(), prefix=lens, drafts=np.asarray(n),
                 parents=flat, q=W.bf16_bits(q), k_scale=scales[0] if fp8 else None, v_scale=scales[1] if fp8 else None,
                 pool_k=pool[0].cpu().numpy() if fp8 else W.bf16_bits(pool[0]),
                 pool_v=pool[1].cpu().numpy() if fp8 else W.bf16_bits(pool[1]))
        assert_attention(W.bf16_bits(out), c, f"step {step}")
        a = accept_case(96 + step, drafts=n, V=V, drawn=True)
        a["parents"] = flat
        acc, cnt, nxt = B.sgl_verify_drafts(*[torch.from_numpy(a[k]).to(DEV) for k in
                                              ("p", "tok", "parents", "drafts", "coins", "final", "q")], max_draft=most)
        want = oracle.drafts.verify_drafts(a["p"], a["q"], a["tok"], flat, n, a["coins"], a["final"], most)
        assert np.array_equal(acc.cpu().numpy(), want[0]) and np.array_equal(nxt.cpu().numpy(), want[2])
        seq, freed, count = B.sgl_commit_drafts(rtt, rows, pre, dl, W.int_tensor(slots, DEV), acc, cnt)
        at = 0
        for r in range(b):
            kept_rows[r] += [int(slots[at + i]) for i in want[0][r][: want[1][r]]]
            at += n[r]
        lens = seq.cpu().numpy().astype(np.int32)
        assert lens.tolist() == [len(x) for x in kept_rows]
        free += freed[: int(count.item())].tolist()
        dq = W.bf16_tensor(W.f32_to_bf16_bits(g.standard_normal((b, Hq, D)).astype(np.float32)), DEV)
        decode = getattr(B, "sgl_decode_attention" + tail)
        got = decode(dq, *pool, *scales, rtt, rows, seq, max_seq_len=cap)
        own = torch.zeros_like(rtt)
        for r in range(b):
            own[r, : lens[r]] = torch.tensor(kept_rows[r], dtype=torch.int32, device=DEV)
        ref = decode(dq, *pool, *scales, own, rows, seq, max_seq_len=cap)
        assert torch.equal(got.view(torch.int16), ref.view(torch.int16))
