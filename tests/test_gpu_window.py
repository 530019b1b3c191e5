"""Sliding-window decode and extend against the fp64 oracle, within the bounds
derived in _window.py.  Hidden positions' entries of req_to_token point at NaN
rows, so a key that should not be seen shows up as NaN."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import oracle  # noqa: E402
from radixattention_prefix_shared_gb300 import binding as B  # noqa: E402
from radixattention_prefix_shared_gb300 import workloads as W  # noqa: E402

from _window import assert_within, attention_case, readers  # noqa: E402

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]

DEV = "cuda:0"


class Case:
    """A case's inputs on the GPU and the calls over them."""

    def __init__(self, c):
        self.c = c
        self.q = W.bf16_tensor(c["q"], DEV)
        up = (lambda x: torch.from_numpy(x).to(DEV)) if c["fp8"] else (lambda x: W.bf16_tensor(x, DEV))
        self.pk, self.pv = up(c["pool_k"]), up(c["pool_v"])
        self.rtt, self.rpi, self.prefix, self.ext, self.seq = (
            W.int_tensor(c[n], DEV) for n in ("rtt", "rpi", "prefix", "ext", "seq"))
        self.scales = (c["k_scale"], c["v_scale"]) if c["fp8"] else ()
        self.kw = dict(window=c["window"], sinks=c["sinks"])

    def decode(self, **kw):
        f = B.sgl_decode_attention_window_fp8 if self.c["fp8"] else B.sgl_decode_attention_window
        a = dict(max_seq_len=max(1, int(self.c["seq"].max())), **self.kw)
        a.update(kw)
        return f(self.q, self.pk, self.pv, *self.scales, self.rtt, self.rpi, self.seq, **a)

    def extend(self, **kw):
        f = B.sgl_extend_attention_window_fp8 if self.c["fp8"] else B.sgl_extend_attention_window
        a = dict(max_extend=int(self.c["ext"].max()), max_prefix=int(self.c["prefix"].max()), **self.kw)
        a.update(kw)
        return f(self.q, self.pk, self.pv, *self.scales, self.rtt, self.rpi, self.prefix, self.ext, **a)

    def want_decode(self):
        c = self.c
        return oracle.window.decode_attention_window(c["q"], *readers(c), c["rtt"], c["rpi"], c["seq"], c["Hkv"],
                                                     c["window"], c["sinks"])

    def want_extend(self, tokens=None):
        c = self.c
        return oracle.window.extend_attention_window(c["q"], *readers(c), c["rtt"], c["rpi"], c["prefix"], c["ext"],
                                                     c["Hkv"], c["window"], c["sinks"], tokens=tokens)


def decode_case(seed, seq, **kw):
    """One query a request; requests of length 0 keep a (padding) query row."""
    ext = [1 if n > 0 else 0 for n in seq]
    c = attention_case(seed, prefix=[max(0, n - 1) for n in seq], ext=ext, **kw)
    g = np.random.default_rng(seed + 1)
    c["q"] = W.f32_to_bf16_bits(g.standard_normal((len(seq), c["Hq"], c["D"])).astype(np.float32))
    return Case(c)


def check_decode(case, out, what=""):
    live = case.c["seq"] > 0
    return assert_within(W.bf16_bits(out), *case.want_decode(), case.c["fp8"], rows=live, what=what)


# ------------------------------------------------------------------ decode

HEADS = [(1, 1, 64), (4, 4, 128), (16, 8, 128), (12, 4, 64), (8, 2, 128), (5, 1, 128), (16, 2, 64), (18, 2, 128),
         (16, 1, 64), (34, 2, 64), (64, 2, 128), (6, 3, 128)]
# around sinks + window, the split kernel's stages and one key
LENS = [1, 2, 9, 10, 11, 12, 13, 31, 32, 33, 64, 65, 200, 0, 517]


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("heads", HEADS, ids=lambda h: f"{h[0]}q{h[1]}kv{h[2]}d")
def test_decode_head_layouts(heads, fp8):
    Hq, Hkv, D = heads
    for window, sinks in ((9, 3), (64, 0)):
        case = decode_case(Hq + D, LENS, Hq=Hq, Hkv=Hkv, D=D, window=window, sinks=sinks, fp8=fp8)
        check_decode(case, case.decode(), f"{heads} window {window}")


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (2, 5), (7, 1), (100, 100), (600, 0), (1500, 4), (4096, 4),
                                          (3, 1000), (2**31 - 1, 0), (2**31 - 1, 2**31 - 1)])
def test_decode_windows(window, sinks, fp8):
    case = decode_case(window % 97, [1, 6, 101, 2500, 5000], Hq=8, Hkv=4, D=128, window=window, sinks=sinks, fp8=fp8)
    check_decode(case, case.decode(), f"window {window} sinks {sinks}")


# as many requests as fill the device with one CTA a group of 4 KV heads: rows
# of at most 128 bytes are gathered in spans there; one run a request, and many
@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("shape", [(16, 16, 64, 70, 100, 3), (16, 16, 128, 66, 250, 0), (32, 16, 64, 65, 40, 1),
                                   (64, 16, 64, 16, 1000, 5), (48, 16, 64, 18, 800, 0), (80, 16, 64, 17, 900, 2),
                                   (32, 16, 128, 16, 1000, 1), (32, 8, 64, 16, 2000, 4), (112, 16, 64, 16, 1021, 0)],
                         ids=lambda s: f"{s[0]}q{s[1]}kv{s[2]}d_b{s[3]}_w{s[4]}")
def test_decode_of_many_requests(shape, fp8):
    Hq, Hkv, D, batch, window, sinks = shape
    g = np.random.default_rng(batch)
    seq = [int(n) for n in g.integers(1, window + window // 2, batch)]
    seq[:5] = [1, 0, window, window + sinks, window + sinks + 1]
    case = decode_case(Hq + window, seq, Hq=Hq, Hkv=Hkv, D=D, window=window, sinks=sinks, fp8=fp8)
    check_decode(case, case.decode(max_seq_len=2 * window), f"{shape}")


def test_decode_full_window_equals_decode():
    """With a window over everything the call is sgl_decode_attention."""
    case = decode_case(11, [700, 1, 33, 2048], Hq=16, Hkv=8, D=128, window=5000, sinks=0)
    got = case.decode()
    plain = B.sgl_decode_attention(case.q, case.pk, case.pv, case.rtt, case.rpi, case.seq, max_seq_len=2048)
    check_decode(case, got)
    check_decode(case, plain)


def test_decode_padding_rows_are_left_alone():
    case = decode_case(12, [0, 40, -3, 0, 7], Hq=8, Hkv=2, D=64, window=16, sinks=2)
    case.seq = W.int_tensor(np.array([0, 40, -3, 0, 7], np.int32), DEV)
    out = torch.full_like(case.q, 7.25)
    case.decode(out=out)
    check_decode(case, out)
    assert (out[[0, 2, 3]] == 7.25).all()


def test_decode_lengths_above_the_host_maximum_read_nothing_past_it():
    """seq_lens above max_seq_len: keys past it are never read (the call stays in bounds)."""
    case = decode_case(13, [50, 60], Hq=8, Hkv=2, D=64, window=20, sinks=2)
    case.c["seq"] = np.array([50, 50], np.int32)
    case2 = decode_case(13, [50, 60], Hq=8, Hkv=2, D=64, window=100, sinks=2)
    out = case2.decode(max_seq_len=50)
    case2.c["seq"] = np.array([50, 50], np.int32)
    check_decode(case2, out)


def test_decode_wide_scores_and_sinks_that_take_the_weight():
    for fp8 in (False, True):
        case = decode_case(14, [900, 2000], Hq=8, Hkv=4, D=128, window=800, sinks=4, fp8=fp8, std=4.0)
        check_decode(case, case.decode(), "wide scores")


# ------------------------------------------------------------------ extend

EXTENDS = [
    # (Hq, Hkv, D, prefix, ext, window, sinks)
    (2, 2, 64, [0, 16, 33, 64], [8, 1, 31, 17], 10, 2),
    (4, 4, 128, [0, 127, 128, 129], [1, 128, 129, 300], 128, 4),
    (8, 2, 128, [300, 5, 0], [64, 65, 200], 1, 0),
    (16, 8, 128, [1, 513], [257, 33], 100, 0),
    (16, 2, 64, [40, 0, 700], [9, 0, 31], 256, 300),
    (8, 1, 128, [1290], [140], 500, 1),
    (6, 2, 128, [70, 3], [50, 90], 20, 130),     # g = 3: padding rows in the tiles
    (32, 1, 64, [64, 7], [33, 20], 5, 3),        # g = 32: 4 tokens a tile
    (34, 2, 64, [200], [11], 64, 4),             # g = 17
    (256, 2, 64, [20], [3], 7, 1),               # g = 128: one token a tile
    (8, 8, 128, [100], [700], 300, 4),           # g = 1: 256 tokens a CTA
]


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("shape", EXTENDS, ids=lambda s: f"{s[0]}q{s[1]}kv{s[2]}d_w{s[5]}s{s[6]}")
def test_extend_matches_oracle(shape, fp8):
    Hq, Hkv, D, prefix, ext, window, sinks = shape
    case = Case(attention_case(Hq + window, Hq=Hq, Hkv=Hkv, D=D, prefix=prefix, ext=ext, window=window, sinks=sinks,
                               fp8=fp8))
    assert_within(W.bf16_bits(case.extend()), *case.want_extend(), fp8, what=str(shape))


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("window,sinks", [(1, 1), (127, 1), (128, 0), (129, 5), (2000, 4), (2**31 - 1, 0),
                                          (50, 2**31 - 1)])
def test_extend_windows_across_blocks(window, sinks, fp8):
    case = Case(attention_case(window % 91, Hq=4, Hkv=2, D=128, prefix=[900, 0], ext=[300, 261], window=window,
                               sinks=sinks, fp8=fp8))
    tokens = [0, 1, 63, 64, 127, 128, 200, 299, 300, 301, 427, 428, 560]
    want, terms = case.want_extend(tokens)
    assert_within(W.bf16_bits(case.extend()), want, terms, fp8, rows=tokens)


# (Hq, Hkv, D, requests, window, sinks, longest extend): enough tiles for every
# SM, so that no tile's keys are dealt to several CTAs (the shapes above are
# dealt); requests of one Q tile, of two with few keys (one tile a CTA over
# bf16 pools) and of two with many (two tiles a CTA)
MANY = [(16, 16, 64, 12, 200, 3, 25), (40, 20, 128, 9, 70, 0, 25), (96, 32, 64, 5, 300, 130, 25),
        (40, 40, 64, 5, 90, 2, 150), (80, 40, 128, 4, 100, 0, 100), (40, 40, 64, 5, 600, 4, 150),
        (80, 40, 128, 4, 500, 20, 100)]


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("shape", MANY, ids=lambda s: f"{s[0]}q{s[1]}kv{s[2]}d_w{s[4]}_e{s[6]}")
def test_extend_of_many_tiles(shape, fp8):
    Hq, Hkv, D, n, window, sinks, longest = shape
    g = np.random.default_rng(n)
    ext = g.integers(0, longest, n).tolist()
    ext[1] = longest - 1
    case = Case(attention_case(n, Hq=Hq, Hkv=Hkv, D=D, prefix=g.integers(0, 800, n).tolist(), ext=ext, window=window,
                               sinks=sinks, fp8=fp8))
    total = sum(ext)
    picked = {0, ext[0], ext[0] + 63, ext[0] + longest - 2, total - 1} | set(g.integers(0, total, 12).tolist())
    tokens = sorted(t for t in picked if t < total)
    out = case.extend()
    assert torch.isfinite(out).all()
    assert_within(W.bf16_bits(out), *case.want_extend(tokens), fp8, rows=tokens, what=str(shape))


def test_extend_full_window_equals_extend():
    """With a window over everything the call is sgl_extend_attention over the stored suffix."""
    case = Case(attention_case(21, Hq=8, Hkv=4, D=128, prefix=[130, 0], ext=[70, 200], window=1000, sinks=0))
    c = case.c
    new = np.concatenate([c["rtt"][c["rpi"][r], p: p + e] for r, (p, e) in enumerate(zip(c["prefix"], c["ext"]))])
    k_new, v_new = (W.bf16_tensor(c[n][new], DEV) for n in ("pool_k", "pool_v"))
    plain = B.sgl_extend_attention(case.q, k_new, v_new, case.pk, case.pv, case.rtt, case.rpi, case.prefix, case.ext,
                                   max_extend=200, max_prefix=130)
    want = case.want_extend()
    assert_within(W.bf16_bits(plain), *want, False)
    assert_within(W.bf16_bits(case.extend()), *want, False)


def test_extend_rows_past_the_suffixes_are_left_alone():
    case = Case(attention_case(22, Hq=4, Hkv=2, D=64, prefix=[5, 9], ext=[6, 3], window=4, sinks=1))
    q = torch.cat([case.q, torch.zeros_like(case.q[:5])])
    case.q = q
    out = torch.full_like(q, -3.5)
    case.extend(out=out, total_extend=9)
    want, terms = case.want_extend()
    assert_within(W.bf16_bits(out[:9]), want, terms, False)
    assert (out[9:] == -3.5).all()
    # a padded batch: total_extend counts rows behind the last request (few
    # tiles of many keys, dealt to several CTAs; then few keys)
    for window in (700, 4):
        case = Case(attention_case(25, Hq=4, Hkv=2, D=64, prefix=[900, 9], ext=[6, 3], window=window, sinks=1))
        case.q = torch.cat([case.q, torch.zeros(3000, 4, 64, dtype=torch.bfloat16, device=DEV)])
        out = torch.full_like(case.q, -3.5)
        case.extend(out=out, total_extend=3009)
        want, terms = case.want_extend()
        assert_within(W.bf16_bits(out[:9]), want, terms, False)
        assert (out[9:] == -3.5).all()


def test_extend_wide_scores():
    for fp8 in (False, True):
        case = Case(attention_case(23, Hq=4, Hkv=2, D=128, prefix=[400], ext=[140], window=300, sinks=4, fp8=fp8,
                                   std=4.0))
        assert_within(W.bf16_bits(case.extend()), *case.want_extend(), fp8)


def test_single_tokens_of_extend_and_decode_agree_with_each_other():
    for fp8 in (False, True):
        case = Case(attention_case(24, Hq=16, Hkv=8, D=128, prefix=[2000, 17, 0], ext=[1, 1, 1], window=600, sinks=4,
                                   fp8=fp8))
        want, terms = case.want_extend()
        assert_within(W.bf16_bits(case.extend()), want, terms, fp8)
        assert_within(W.bf16_bits(case.decode()), want, terms, fp8)


# ------------------------------------------------------------------ index checks

def _kind(call):
    err = torch.zeros(4, dtype=torch.int32, device=DEV)
    call(err)
    torch.cuda.synchronize()
    return err.tolist()


def test_checks_read_what_the_calls_read():
    case = Case(attention_case(31, Hq=2, Hkv=2, D=64, prefix=[40, 0], ext=[6, 4], window=8, sinks=3))
    S = case.c["S"]
    row = case.c["rpi"][0]
    seq = W.int_tensor(np.array([46, 0], np.int32), DEV)

    def ext(err, rtt):
        B.sgl_check_extend_window_indices(rtt, case.rpi, case.prefix, case.ext, total_extend=10, max_extend=6,
                                          max_prefix=40, window=8, sinks=3, pool_size=S, d_error=err)

    def dec(err, rtt, seq=seq):
        B.sgl_check_decode_window_indices(rtt, case.rpi, seq, max_seq_len=46, window=8, sinks=3, pool_size=S,
                                          d_error=err)
    good = case.rtt.clone()
    good[row, 3:33] = -1                     # hidden from the extend's first query on
    assert _kind(lambda e: ext(e, good))[0] == 0
    for j in (0, 2, 33, 45):
        bad = good.clone()
        bad[row, j] = S
        assert _kind(lambda e: ext(e, bad)) == [1, 0, j, S]
    good[row, 33:38] = -1                    # the decode's query sees 38 .. 45
    assert _kind(lambda e: dec(e, good))[0] == 0
    for j in (1, 38, 45):
        bad = good.clone()
        bad[row, j] = -7
        assert _kind(lambda e: dec(e, bad)) == [1, 0, j, -7]
    assert _kind(lambda e: dec(e, good, W.int_tensor(np.array([46, -1], np.int32), DEV)))[0] == 3


# ------------------------------------------------------------------ the binding's refusals

def test_binding_refuses_what_it_would_misread():
    case = Case(attention_case(32, Hq=4, Hkv=2, D=64, prefix=[9], ext=[1], window=4, sinks=1))
    for attr, bad in (("q", case.q.half()), ("pk", case.pk.float()), ("rtt", case.rtt.long()),
                      ("rpi", case.rpi[:0]), ("q", case.q.cpu()), ("pk", case.pk[:, :, :32]),
                      ("seq", case.seq.long())):
        keep = getattr(case, attr)
        setattr(case, attr, bad)
        with pytest.raises(ValueError):
            case.decode()
        setattr(case, attr, keep)
    with pytest.raises(ValueError):
        case.decode(out=case.q[:, :2])
    with pytest.raises(ValueError):
        case.extend(total_extend=2)
    with pytest.raises(B.SglError):
        case.decode(window=0)
    with pytest.raises(B.SglError):
        case.extend(sinks=-1)
