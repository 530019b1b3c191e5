"""The drafted-token oracle pinned against the other oracles, brute force and the
distribution that the walk is to keep; and the calls' host-side checks."""
import ctypes
import itertools

import numpy as np
import pytest

import oracle
from radixattention_prefix_shared_gb300 import binding as B

from _drafts import attention_case, softmax_rows, tree, want_attention

FAKE = ctypes.c_void_p(0x100000)     # aligned, never dereferenced
MISALIGNED = ctypes.c_void_p(0x100008)


# ------------------------------------------------------------------ attention

@pytest.mark.parametrize("fp8", [False, True])
def test_a_chain_is_an_extend(fp8):
    c = attention_case(1, Hq=4, Hkv=2, D=64, prefix=[0, 9, 40], drafts=[3, 5, 1], kind="chain", fp8=fp8)
    out, _ = want_attention(c)
    read = [oracle.window.pool_reader(c["pool_" + x], c[x + "_scale"]) for x in "kv"]
    ref, _ = oracle.window.extend_attention_window(c["q"], *read, c["rtt"], c["rpi"], c["prefix"], c["drafts"], 2,
                                                   10**6, 0)
    assert np.abs(out - ref).max() < 1e-12


def test_one_node_is_a_decode():
    c = attention_case(2, Hq=4, Hkv=4, D=64, prefix=[0, 7, 30], drafts=[1, 1, 1])
    out, _ = want_attention(c)
    ref = oracle.decode_attention(c["q"], c["pool_k"], c["pool_v"], c["rtt"], c["rpi"], c["prefix"] + 1, 4)
    assert np.abs(out - ref).max() < 1e-12


def test_siblings_do_not_see_each_other():
    """A node sees what it would see were its line of ancestors the whole chain."""
    c = attention_case(3, Hq=2, Hkv=1, D=64, prefix=[11], drafts=[9], kind="tree")
    out, _ = want_attention(c)
    for i in range(9):
        line = oracle.drafts.line_of(c["parents"], i)
        row = np.concatenate([c["rtt"][c["rpi"][0], :11], c["rtt"][c["rpi"][0], 11 + np.asarray(line)]])
        ref = oracle.decode_attention(c["q"][i: i + 1], c["pool_k"], c["pool_v"], row[None], [0], [11 + len(line)], 1)
        assert np.abs(out[i] - ref[0]).max() < 1e-12


def test_lines():
    assert oracle.drafts.line_of([-1, 0, 0, 2, -1, 9, 6], 3) == [0, 2, 3]
    assert [oracle.drafts.line_of([-1, 0, 0, 2, -1, 9, 6], i) for i in (4, 5, 6)] == [[4], [5], [6]]
    g = np.random.default_rng(0)
    for kind in ("chain", "bush", "tree", "forest"):
        par = tree(g, 20, kind)
        for i in range(20):
            line = oracle.drafts.line_of(par, i)
            assert line[-1] == i and all(par[b] == a for a, b in zip(line, line[1:])) and par[line[0]] == -1


# ------------------------------------------------------------------ the walk

def _first_token(target, draft, tokens, parents, coins, final):
    kept, nxt = oracle.drafts.walk(target, draft, tokens, parents, coins, final)
    return int(tokens[kept[1]]) if len(kept) > 1 else nxt


@pytest.mark.parametrize("drawn", [True, False])
def test_the_first_token_keeps_the_targets_distribution(drawn):
    """Three children of the root, drawn with replacement from the draft row (or
    picked): over the coins, and the draws, the first token is distributed as the
    target row.  30,000 walks; a frequency is off by 5 sigma <= 5 * 0.5 / sqrt(30,000)
    = 0.0145 with probability 6e-7."""
    g = np.random.default_rng(5)
    V, walks = 6, 30000
    p, base = softmax_rows(g, 4, V, std=1.0)
    q, _ = softmax_rows(g, 4, V, base=base)
    seen = np.zeros(V)
    picked = np.array([0, 2, 1, 2])
    for _ in range(walks):
        tok = np.concatenate([[0], g.choice(V, size=3, p=q[0] / q[0].sum())]) if drawn else picked
        seen[_first_token(p, q if drawn else None, tok, [-1, 0, 0, 0], g.random(4), g.random())] += 1
    assert np.abs(seen / walks - p[0]).max() < 0.0145


def test_one_draft_by_measure():
    """One drawn child: it is kept for coins below p/q, exactly, and what is left is
    max(p - q, 0)."""
    g = np.random.default_rng(6)
    p, base = softmax_rows(g, 2, 5, std=1.0)
    q, _ = softmax_rows(g, 2, 5, base=base)
    p64, q64 = p.astype(np.float64), q.astype(np.float64)
    for x in range(5):
        border = p64[0, x] / q64[0, x]
        for u in (0.0, border * (1 - 1e-12), border * (1 + 1e-12), 0.999):
            if u >= 1:
                continue
            kept, nxt = oracle.drafts.walk(p, q, [0, x], [-1, 0], [0.5, u], 0.3)
            assert (len(kept) == 2) == (u * q64[0, x] < p64[0, x])
            row = p64[1] if len(kept) == 2 else np.maximum(p64[0] - q64[0], 0)
            assert nxt == int(np.searchsorted(np.cumsum(row), 0.3 * row.sum(), side="right"))


def test_walk_corner_cases():
    one = np.array([[0.0, 1.0, 0.0]] * 3, np.float32)
    # a token twice among siblings, and one outside the vocabulary
    kept, nxt = oracle.drafts.walk(one, None, [0, 2, 1], [-1, 0, 0], [0, 0, 0.9], 0.5)
    assert (kept, nxt) == ([0, 2], 1)
    kept, nxt = oracle.drafts.walk(one, None, [0, 7, -1], [-1, 0, 0], [0, 0, 0], 0.5)
    assert (kept, nxt) == ([0], 1)
    # nothing is left: the row itself; a row without weights
    kept, nxt = oracle.drafts.walk(one, one, [0, 1], [-1, 0], [0, 1.0], 0.0)
    assert (kept, nxt) == ([0], 1)
    bad = np.array([[np.nan, -1.0, np.inf]], np.float32)
    assert oracle.drafts.walk(bad, None, [0], [-1], [0], 0.5) == ([0], -1)


def test_commit_by_hand():
    table = np.arange(24, dtype=np.int32).reshape(2, 12) + 100
    out, seq, freed = oracle.drafts.commit_drafts(table, [1, 0], [3, 5], [4, 2], [10, 11, 12, 13, 14, 15],
                                                  [[0, 2, -1, -1], [0, 1, -1, -1]], [2, 2])
    assert seq.tolist() == [5, 7] and freed.tolist() == [11, 13]
    assert out[1, 3:5].tolist() == [10, 12] and out[0, 5:7].tolist() == [14, 15]
    same = np.ones_like(table, bool)
    same[1, 3:5] = same[0, 5:7] = False
    assert (out == table)[same].all()


# ------------------------------------------------------------------ host checks

def _dims(**kw):
    return B.make_dims(**(dict(num_q_heads=8, num_kv_heads=4, head_dim=128, pool_size=1000, sm_scale=0.0) | kw))


@pytest.mark.parametrize("fp8", [False, True])
def test_verify_attention_refuses(cuda_lib, fp8):
    d = _dims()
    need = B.verify_workspace_bytes(3, 12, 6, 50, 10, d)

    def call(dims=d, **kw):
        a = dict(q=FAKE, pk=FAKE, pv=FAKE, ks=1.0, vs=1.0, rtt=FAKE, rows=5, stride=64, rpi=FAKE, pre=FAKE, dl=FAKE,
                 par=FAKE, batch=3, total=12, most=6, prefix=50, shared=10, out=ctypes.c_void_p(0x10000000), ws=FAKE,
                 wsb=need)
        a.update(kw)
        f = cuda_lib.sgl_verify_attention_fp8 if fp8 else cuda_lib.sgl_verify_attention
        scales = (a["ks"], a["vs"]) if fp8 else ()
        return f(a["q"], a["pk"], a["pv"], *scales, a["rtt"], a["rows"], a["stride"], a["rpi"], a["pre"], a["dl"],
                 a["par"], a["batch"], a["total"], a["most"], a["prefix"], a["shared"], a["out"], a["ws"], a["wsb"],
                 ctypes.byref(dims) if dims is not None else None, None)

    assert call(batch=0) == 0 and call(total=0, most=0) == 0
    assert call(dims=None) == 1
    assert call(dims=_dims(head_dim=96)) == 2
    assert call(dims=_dims(num_q_heads=6)) == 1
    assert call(dims=_dims(num_q_heads=4 * 129)) == 2
    for name in ("batch", "total", "most", "prefix", "shared"):
        assert call(**{name: -1}) == 1
    assert call(most=65, total=70) == 2            # more nodes than a tree may have
    assert call(most=13) == 1                      # above total_draft
    assert call(most=0) == 1
    assert call(shared=51) == 1                    # above every prefix
    assert call(stride=50) == 1                    # prefixes past the row's end
    assert call(total=2**28) == 2                  # rows past 32 bits
    for name in ("q", "pk", "pv", "rtt", "rpi", "pre", "dl", "par", "out"):
        assert call(**{name: None}) == 1
    for name in ("q", "pk", "pv", "out"):
        assert call(**{name: MISALIGNED}) == 1
    assert call(out=ctypes.c_void_p(FAKE.value + 256)) == 1    # part of q
    assert call(q=ctypes.c_void_p(0x20000000), out=FAKE) == 1  # the pool
    assert call(ws=None) == 3 and call(wsb=need - 1) == 3 and call(ws=MISALIGNED) == 3
    if fp8:
        for bad in (0.0, -1.0, float("inf"), float("nan")):
            assert call(ks=bad) == 1 and call(vs=bad) == 1


def test_workspace_grows_with_every_argument():
    base = dict(batch=2, total_draft=10, max_draft=3, max_prefix=100, shared_len=0)
    grow = dict(batch=[5, 300], total_draft=[11, 4000], max_draft=[8, 9, 40, 64], max_prefix=[5000, 10**6],
                shared_len=[1, 90])
    for Hq, Hkv in ((4, 4), (12, 4), (16, 1)):
        d = _dims(num_q_heads=Hq, num_kv_heads=Hkv)
        for name, values in grow.items():
            for rest in itertools.product([False, True], repeat=2):
                b = dict(base)
                if rest[0]:
                    b["shared_len"] = 50
                if rest[1]:
                    b["max_draft"], b["total_draft"] = 20, 200
                sizes = [B.verify_workspace_bytes(**(b | {name: max(v, b[name])}), dims=d) for v in [b[name]] + values]
                assert sizes == sorted(sizes), (name, sizes)
    for bad in (2**31, -2**31, 2**40):
        for name in base:
            with pytest.raises(ValueError, match=name):
                B.verify_workspace_bytes(**(base | {name: bad}), dims=_dims())


def test_verify_drafts_refuses(cuda_lib):
    def call(**kw):
        a = dict(p=FAKE, pst=100, q=FAKE, qst=100, V=100, tok=FAKE, par=FAKE, dl=FAKE, batch=3, total=12, most=6,
                 coins=FAKE, final=FAKE, acc=FAKE, num=FAKE, nxt=FAKE)
        a.update(kw)
        return cuda_lib.sgl_verify_drafts(a["p"], a["pst"], a["q"], a["qst"], a["V"], a["tok"], a["par"], a["dl"],
                                          a["batch"], a["total"], a["most"], a["coins"], a["final"], a["acc"],
                                          a["num"], a["nxt"], None)
    assert call(batch=0) == 0
    for name in ("batch", "total", "most"):
        assert call(**{name: -1}) == 1
    assert call(V=0) == 1 and call(pst=99) == 1 and call(qst=99) == 1
    assert call(most=65) == 2 and call(V=2**30 + 1, pst=2**31, qst=2**31) == 2 and call(most=0) == 1
    for name in ("p", "tok", "par", "dl", "coins", "final", "acc", "num", "nxt"):
        assert call(**{name: None}) == 1


def test_commit_refuses(cuda_lib):
    def call(**kw):
        a = dict(rtt=FAKE, rows=4, stride=20, rpi=FAKE, pre=FAKE, dl=FAKE, slots=FAKE, acc=FAKE, num=FAKE, batch=3,
                 total=12, most=6, seq=FAKE, freed=FAKE, nf=FAKE)
        a.update(kw)
        return cuda_lib.sgl_commit_drafts(a["rtt"], a["rows"], a["stride"], a["rpi"], a["pre"], a["dl"], a["slots"],
                                          a["acc"], a["num"], a["batch"], a["total"], a["most"], a["seq"],
                                          a["freed"], a["nf"], None)
    for name in ("batch", "total", "most"):
        assert call(**{name: -1}) == 1
    assert call(rows=0) == 1 and call(stride=0) == 1 and call(most=65) == 2 and call(most=0) == 1
    for name in ("rtt", "rpi", "pre", "dl", "slots", "acc", "num", "seq", "freed", "nf"):
        assert call(**{name: None}) == 1


def test_check_refuses(cuda_lib):
    def call(**kw):
        a = dict(shared=0, parents=FAKE, err=FAKE, pool=100)
        a.update(kw)
        return cuda_lib.sgl_check_verify_indices(FAKE, 4, 20, FAKE, FAKE, FAKE, a["parents"], 3, 12, 6, 10,
                                                 a["shared"], a["pool"], a["err"], None)
    assert call(shared=-1) == 1 and call(shared=11) == 1 and call(parents=None) == 1 and call(err=None) == 1
    assert call(pool=0) == 1
