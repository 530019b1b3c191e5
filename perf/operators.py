"""Cases of the sliding-window layer step: what a serving loop calls once per
layer of a model whose attention sees a window of recent tokens and a few
first ones.

  rope    head norms of Q and K, rotary positions, K and V stored in the pool
  decode  one query a request over its window and sink tokens
  extend  a chunk of new tokens a request over window and sink tokens

Each case is a dict of plain values; ``prepare`` makes its inputs on the GPU,
``run`` makes one pass (the framework's call where ``own`` is true, elementary
torch operations in 32 bits elsewhere) and ``exact`` computes the same outputs
from the definition in 64 bits.
"""
import math
import random

import torch

own = False
DEV = "cuda"


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one step of 64 decoding requests, 16 query / 8 KV heads of 128
        dict(name="rope_step_64", op="rope", n=64, hq=16, hkv=8, d=128, rot=128, interleaved=False, axes=1,
             norm=True, fp8=False, max_pos=32768),
        # a chunked-prefill step: 8 chunks of 2,048 tokens
        dict(name="rope_prefill_16k", op="rope", n=16384, hq=16, hkv=8, d=128, rot=128, interleaved=False,
             axes=1, norm=True, fp8=False, max_pos=18432),
        # a ragged prefill into an e4m3 pool: half the head rotated, adjacent pairs, no norms, far positions
        dict(name="rope_prefill_fp8_far", op="rope", n=8191, hq=32, hkv=8, d=128, rot=64, interleaved=True,
             axes=1, norm=False, fp8=True, max_pos=1 << 20),
        # a video prompt: time, height and width positions, heads of 64
        dict(name="rope_video_3axes", op="rope", n=4099, hq=16, hkv=4, d=64, rot=64, interleaved=False, axes=3,
             norm=True, fp8=False, max_pos=4096),
        # one interactive request far into its context
        dict(name="decode_single_32k", op="decode", seq_lo=32768, seq_hi=32768, b=1, hq=32, hkv=8, d=128, window=4096,
             sinks=4, fp8=False, lens_seed=1),
        # 248 long multi-turn decodes
        dict(name="decode_248_window_4k", op="decode", seq_lo=1024, seq_hi=32768, b=248, hq=16, hkv=8, d=128,
             window=4096, sinks=4, fp8=False, lens_seed=2),
        # one KV head a query head over an e4m3 pool
        dict(name="decode_64_mha_fp8", op="decode", seq_lo=512, seq_hi=4096, b=64, hq=32, hkv=32, d=128, window=1024,
             sinks=4, fp8=True, lens_seed=3),
        # short odd window, three query heads a KV head, heads of 64
        dict(name="decode_96_window_511", op="decode", seq_lo=1, seq_hi=4096, b=96, hq=12, hkv=4, d=64, window=511,
             sinks=1, fp8=False, lens_seed=4),
        # a short follow-up turn after a long context
        dict(name="extend_turn_37", op="extend", prefix_lo=16001, prefix_hi=16001, ext_lo=37, ext_hi=37, b=1, hq=16, hkv=8, d=128,
             window=1024, sinks=4, fp8=False, lens_seed=5),
        # chunked prefill: 8 chunks of 2,048 tokens after cached prefixes
        dict(name="extend_chunks_8x2048", op="extend", prefix_lo=0, prefix_hi=16384, ext_lo=2048, ext_hi=2048, b=8, hq=16, hkv=8,
             d=128, window=4096, sinks=4, fp8=False, lens_seed=6),
        # the same traffic over an e4m3 pool, window below the 4,096-token prompt, no sinks
        dict(name="extend_prompt_fp8", op="extend", prefix_lo=4096, prefix_hi=4096, ext_lo=256, ext_hi=256, b=64, hq=32, hkv=8,
             d=128, window=2048, sinks=0, fp8=True, lens_seed=7),
        # ragged short extends of several requests, window shorter than a chunk
        dict(name="extend_ragged_17", op="extend", prefix_lo=0, prefix_hi=2000, ext_lo=1, ext_hi=700, b=17, hq=8, hkv=2, d=64,
             window=200, sinks=3, fp8=False, lens_seed=8),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "decode", "decode", "extend", "extend"])
    d = rng.choice([64, 128, 128])
    hkv = rng.choice([1, 2, 3, 4, 8, 8])
    g = rng.choice([1, 2, 2, 3, 4, 4, 5, 8])
    fp8 = rng.random() < 0.4
    if op == "rope":
        rot = rng.choice([d, d, d // 2, 16, 48])
        return dict(op=op, n=_log_int(rng, 1, 10000), hq=min(32, hkv * g) // hkv * hkv, hkv=hkv, d=d, rot=rot,
                    interleaved=rng.random() < 0.4, axes=rng.choice([1, 1, 3]), norm=rng.random() < 0.75,
                    fp8=fp8, max_pos=_log_int(rng, 64, 1 << 20))
    window = _log_int(rng, 1, 4000)
    sinks = rng.choice([0, 1, 4, 4, 16, 100])
    if op == "decode":
        b = _log_int(rng, 1, 200)
        hi = _log_int(rng, 16, 32768)
        return dict(op=op, seq_lo=max(1, hi // rng.choice([1, 4, 32])), seq_hi=hi, b=b, hq=hkv * g, hkv=hkv, d=d,
                    window=window, sinks=sinks, fp8=fp8, lens_seed=rng.randrange(1 << 30))
    ext = _log_int(rng, 1, 2048)
    b = max(1, min(_log_int(rng, 1, 64), 8192 // ext))
    pre = _log_int(rng, 1, 16384)
    return dict(op=op, prefix_lo=0, prefix_hi=pre, ext_lo=max(1, ext // rng.choice([1, 3])), ext_hi=ext, b=b,
                hq=min(32, hkv * g) // hkv * hkv, hkv=hkv, d=d, window=min(window, 3500), sinks=sinks, fp8=fp8, lens_seed=rng.randrange(1 << 30))


def _lens(case, key):
    """The case's lengths: log-uniform over decode ranges, uniform over extend ranges."""
    rng = random.Random(case["lens_seed"] * 7 + len(key))
    lo, hi = case[key + "_lo"], case[key + "_hi"]
    if case["op"] == "decode":
        return [lo if lo == hi else _log_int(rng, lo, hi) for _ in range(case["b"])]
    return [rng.randint(lo, hi) for _ in range(case["b"])]


def _pairs(prefix, ext, window, sinks):
    """Visible (query, key) pairs of one request and the keys some query sees."""
    total = 0
    for p in range(prefix, prefix + ext):
        lo = max(0, p - window + 1)
        total += p + 1 - lo + min(sinks, lo)
    lo = max(0, prefix - window + 1)
    return total, prefix + ext - lo + min(sinks, lo)


def work(case):
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    es = 1 if case["fp8"] else 2
    if case["op"] == "rope":
        n = case["n"]
        return {"bytes": n * d * (2 * hq + 4 * hkv) + n * d * (2 * hq + 2 * hkv * es) + n * 4 * (1 + case["axes"]),
                "flops": n * d * ((5 if case["norm"] else 0) * (hq + hkv) + 4 * (hq + hkv) * case["rot"] // d)}
    if case["op"] == "decode":
        keys = sum(min(x, case["window"] + case["sinks"]) for x in _lens(case, "seq"))
        return {"bytes": keys * (2 * hkv * d * es + 4) + 4 * case["b"] * hq * d, "flops": 4 * d * hq * keys}
    pairs = keys = tokens = 0
    for p, e in zip(_lens(case, "prefix"), _lens(case, "ext")):
        a, b = _pairs(p, e, case["window"], case["sinks"])
        pairs, keys, tokens = pairs + a, keys + b, tokens + e
    return {"bytes": keys * (2 * hkv * d * es + 4) + 4 * tokens * hq * d, "flops": 4 * d * hq * pairs}


# ------------------------------------------------------------------ inputs

def _randn(gen, *shape, std=1.0):
    x = torch.randn(*shape, generator=gen, device=DEV, dtype=torch.bfloat16)
    return x if std == 1.0 else x * std


def _codes(x, scale):
    """e4m3 codes of bf16 rows, saturating."""
    q = (x.float() / scale).clamp_(-448.0, 448.0)
    return q.to(torch.float8_e4m3fn).view(torch.uint8)


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    return _prepare_rope(case, gen) if case["op"] == "rope" else _prepare_attention(case, gen)


def _prepare_rope(case, gen):
    n, hq, hkv, d, rot, axes = (case[k] for k in ("n", "hq", "hkv", "d", "rot", "axes"))
    s = dict(case=case)
    # the projection's packed output: Q, K and V of a token side by side
    s["qkv"] = _randn(gen, n, hq + 2 * hkv, d, std=1.5)
    s["q"], s["k"], s["v"] = s["qkv"].split([hq, hkv, hkv], dim=1)
    s["qw"] = 1 + _randn(gen, d, std=0.2) if case["norm"] else None
    s["kw"] = 1 + _randn(gen, d, std=0.2) if case["norm"] else None
    s["inv_freq"] = (1e6 ** (-torch.arange(0, rot, 2, device=DEV, dtype=torch.float64) / rot)).float()
    pos = torch.randint(0, case["max_pos"], (axes, n), generator=gen, device=DEV, dtype=torch.int32)
    s["positions"] = pos if axes > 1 else pos[0].contiguous()
    # the frequencies of the axes: a quarter for time, the rest split evenly
    nf = rot // 2
    s["freq_axis"] = None
    if axes > 1:
        s["freq_axis"] = torch.tensor([0 if i < nf // 4 else 1 + (i - nf // 4) * (axes - 1) // (nf - nf // 4)
                                       for i in range(nf)], dtype=torch.int32, device=DEV)
    pool = 2 * n + 64
    s["slots"] = torch.randperm(pool, generator=gen, device=DEV)[:n].to(torch.int32)
    s["pool_k"], s["pool_v"] = _randn(gen, pool, hkv, d), _randn(gen, pool, hkv, d)
    if case["fp8"]:
        s["k_scale"], s["v_scale"] = 0.03, 0.02
        s["pool_k"], s["pool_v"] = _codes(s["pool_k"], 0.03), _codes(s["pool_v"], 0.02)
    s["q_out"] = torch.empty(n, hq, d, dtype=torch.bfloat16, device=DEV)
    return s


def _prepare_attention(case, gen):
    hq, hkv, d, b = (case[k] for k in ("hq", "hkv", "d", "b"))
    window, sinks = case["window"], case["sinks"]
    s = dict(case=case)
    if case["op"] == "decode":
        ext = [1] * b
        prefix = [x - 1 for x in _lens(case, "seq")]
    else:
        prefix, ext = _lens(case, "prefix"), _lens(case, "ext")
    seq = [p + e for p, e in zip(prefix, ext)]
    # positions some query sees; the slots of the others were given back and
    # serve other requests by now, so those entries are stale
    spans = []
    for p, e in zip(prefix, ext):
        lo = max(0, p - window + 1)
        spans.append((min(sinks, lo), lo, p + e))
    live = sum(a + z - lo for a, lo, z in spans)
    pool = live + live // 8 + 64
    perm = torch.randperm(pool, generator=gen, device=DEV).to(torch.int32)
    rows, stride = b + 3, max(seq) + 5
    s["req_to_token"] = torch.randint(0, pool, (rows, stride), generator=gen, device=DEV, dtype=torch.int32)
    rpi = list(range(rows))
    random.Random(case["lens_seed"]).shuffle(rpi)
    s["req_pool_idx"] = torch.tensor(rpi[:b], dtype=torch.int32, device=DEV)
    s["pool_k"], s["pool_v"] = _randn(gen, pool, hkv, d), _randn(gen, pool, hkv, d)
    # the first tokens draw a good part of every query's weight
    lead = _randn(gen, hkv, 1, d)
    at = 0
    for r, (a, lo, z) in enumerate(spans):
        row = s["req_to_token"][rpi[r]]
        row[:a] = perm[at: at + a]
        row[lo:z] = perm[at + a: at + a + z - lo]
        first = row[:min(sinks, z)].long()
        s["pool_k"][first] += (0.9 * lead[:, 0]).to(torch.bfloat16)
        at += a + z - lo
    if case["fp8"]:
        s["k_scale"], s["v_scale"] = 0.02, 0.0173
        s["pool_k"], s["pool_v"] = _codes(s["pool_k"], s["k_scale"]), _codes(s["pool_v"], s["v_scale"])
    tokens = sum(ext)
    q = _randn(gen, tokens, hkv, hq // hkv, d) + 0.7 * lead
    s["q"] = q.reshape(tokens, hq, d).contiguous()
    s["out"] = torch.empty_like(s["q"])
    s["prefix"], s["ext"], s["seq"] = prefix, ext, seq
    s["prefix_lens"] = torch.tensor(prefix, dtype=torch.int32, device=DEV)
    s["extend_lens"] = torch.tensor(ext, dtype=torch.int32, device=DEV)
    s["seq_lens"] = torch.tensor(seq, dtype=torch.int32, device=DEV)
    if own:
        from radixattention_prefix_shared_gb300 import binding as B
        dims = B.make_dims(hq, hkv, d, pool)
        if case["op"] == "decode":
            nbytes = B.decode_window_workspace_bytes(b, max(seq), window, sinks, dims)
        else:
            nbytes = B.extend_window_workspace_bytes(b, tokens, max(ext), max(prefix), window, sinks, dims)
        s["workspace"] = B.new_workspace(nbytes, DEV)
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    op = s["case"]["op"]
    if own:
        return {"rope": _own_rope, "decode": _own_decode, "extend": _own_extend}[op](s)
    return {"rope": _plain_rope, "decode": _plain_decode, "extend": _plain_extend}[op](s)


def _rope_outputs(s):
    # an e4m3 pool's rows are returned as the values of their codes
    view = (lambda x: x.view(torch.float8_e4m3fn)) if s["case"]["fp8"] else (lambda x: x)
    return {"q": s["q_out"], "pool_k": view(s["pool_k"]), "pool_v": view(s["pool_v"])}


def _own_rope(s):
    from radixattention_prefix_shared_gb300 import binding as B
    kw = dict(q_weight=s["qw"], k_weight=s["kw"], eps=1e-6, freq_axis=s["freq_axis"],
              interleaved=s["case"]["interleaved"], q_out=s["q_out"])
    if s["case"]["fp8"]:
        B.sgl_qk_norm_rope_store_kv_fp8(s["q"], s["k"], s["v"], s["positions"], s["inv_freq"], s["slots"],
                                        s["pool_k"], s["pool_v"], s["k_scale"], s["v_scale"], **kw)
    else:
        B.sgl_qk_norm_rope_store_kv(s["q"], s["k"], s["v"], s["positions"], s["inv_freq"], s["slots"],
                                    s["pool_k"], s["pool_v"], **kw)
    return _rope_outputs(s)


def _own_decode(s):
    from radixattention_prefix_shared_gb300 import binding as B
    c = s["case"]
    kw = dict(out=s["out"], max_seq_len=max(s["seq"]), window=c["window"], sinks=c["sinks"],
              workspace=s["workspace"])
    if c["fp8"]:
        return B.sgl_decode_attention_window_fp8(s["q"], s["pool_k"], s["pool_v"], s["k_scale"], s["v_scale"],
                                                 s["req_to_token"], s["req_pool_idx"], s["seq_lens"], **kw)
    return B.sgl_decode_attention_window(s["q"], s["pool_k"], s["pool_v"], s["req_to_token"],
                                         s["req_pool_idx"], s["seq_lens"], **kw)


def _own_extend(s):
    from radixattention_prefix_shared_gb300 import binding as B
    c = s["case"]
    kw = dict(out=s["out"], max_extend=max(s["ext"]), max_prefix=max(s["prefix"]), window=c["window"],
              sinks=c["sinks"], workspace=s["workspace"])
    if c["fp8"]:
        return B.sgl_extend_attention_window_fp8(s["q"], s["pool_k"], s["pool_v"], s["k_scale"], s["v_scale"],
                                                 s["req_to_token"], s["req_pool_idx"], s["prefix_lens"],
                                                 s["extend_lens"], **kw)
    return B.sgl_extend_attention_window(s["q"], s["pool_k"], s["pool_v"], s["req_to_token"],
                                         s["req_pool_idx"], s["prefix_lens"], s["extend_lens"], **kw)


# ------------------------------------------------------------------ plain forms

def _plain_rope(s):
    c = s["case"]
    rot, slots = c["rot"], s["slots"].long()
    pos = s["positions"].double()
    if c["axes"] > 1:
        ang = pos[s["freq_axis"].long()].T * s["inv_freq"].double()
    else:
        ang = pos[:, None] * s["inv_freq"].double()
    cos, sin = torch.cos(ang).float()[:, None], torch.sin(ang).float()[:, None]

    def turn(x, w):
        y = x.float()
        if w is not None:
            y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + 1e-6) * w.float()
        if c["interleaved"]:
            a, b = y[..., 0:rot:2], y[..., 1:rot:2]
            r = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
        else:
            a, b = y[..., : rot // 2], y[..., rot // 2: rot]
            r = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
        return torch.cat((r, y[..., rot:]), -1)

    s["q_out"].copy_(turn(s["q"], s["qw"]))
    k, v = turn(s["k"], s["kw"]), s["v"]
    if c["fp8"]:
        s["pool_k"][slots] = _codes(k, s["k_scale"])
        s["pool_v"][slots] = _codes(v, s["v_scale"])
    else:
        s["pool_k"][slots] = k.to(torch.bfloat16)
        s["pool_v"][slots] = v
    return _rope_outputs(s)


def _rows(s, which, slots):
    x = s["pool_" + which][slots]
    return x.view(torch.float8_e4m3fn).float() * s[which + "_scale"] if s["case"]["fp8"] else x.float()


def _plain_decode(s):
    c = s["case"]
    hkv, d, b = c["hkv"], c["d"], c["b"]
    seq = s["seq_lens"].long()[:, None]
    most = min(max(s["seq"]), c["window"] + c["sinks"])
    j = torch.arange(most, device=DEV)[None]
    n = torch.clamp(seq, max=c["window"] + c["sinks"])
    pos = torch.where(j < c["sinks"], j, j + (seq - n))
    seen = j < n
    slots = torch.gather(s["req_to_token"][s["req_pool_idx"].long()].long(), 1, torch.where(seen, pos, 0))
    q = s["q"].float().view(b, hkv, -1, d)
    sc = torch.einsum("bhgd,bjhd->bhgj", q, _rows(s, "k", slots)) / math.sqrt(d)
    sc = sc.masked_fill(~seen[:, None, None], float("-inf"))
    p = torch.exp(sc - sc.amax(-1, keepdim=True))
    o = torch.einsum("bhgj,bjhd->bhgd", p, _rows(s, "v", slots)) / p.sum(-1, keepdim=True)
    s["out"].copy_(o.reshape(b, -1, d))
    return s["out"]


def _plain_extend(s):
    c = s["case"]
    hkv, d, window, sinks = c["hkv"], c["d"], c["window"], c["sinks"]
    rpi, at = s["req_pool_idx"].long(), 0
    for r, (p, e) in enumerate(zip(s["prefix"], s["ext"])):
        lo = max(0, p - window + 1)
        pos = torch.cat((torch.arange(min(sinks, lo), device=DEV), torch.arange(lo, p + e, device=DEV)))
        slots = s["req_to_token"][rpi[r]][pos].long()
        k, v = _rows(s, "k", slots).transpose(0, 1)[:, None], _rows(s, "v", slots).transpose(0, 1)[:, None]
        me = torch.arange(p, p + e, device=DEV)[:, None]
        seen = (pos <= me) & ((pos < sinks) | (pos > me - window))
        q = s["q"][at: at + e].float().view(e, hkv, -1, d).permute(1, 2, 0, 3)
        sc = (q @ k.transpose(-1, -2)) / math.sqrt(d)
        sc = sc.masked_fill(~seen, float("-inf"))
        w = torch.exp(sc - sc.amax(-1, keepdim=True))
        o = (w @ v) / w.sum(-1, keepdim=True)
        s["out"][at: at + e] = o.permute(2, 0, 1, 3).reshape(e, -1, d).to(torch.bfloat16)
        at += e
    return s["out"]


# ------------------------------------------------------------------ 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return _exact_rope(s) if case["op"] == "rope" else _exact_attention(s)


def _exact_rope(s):
    c, d = s["case"], s["case"]["d"]
    rot, nf = c["rot"], c["rot"] // 2
    first = torch.arange(nf, device=DEV) * (2 if c["interleaved"] else 1)
    second = first + (1 if c["interleaved"] else nf)
    axis = s["freq_axis"].long() if c["axes"] > 1 else torch.zeros(nf, dtype=torch.long, device=DEV)
    pos = s["positions"].view(c["axes"], -1).double()
    turn = torch.polar(torch.ones((), dtype=torch.float64, device=DEV),
                       torch.einsum("fn,f->nf", pos[axis], s["inv_freq"].double()))

    def rows(x, w):
        y = x.double()
        if w is not None:
            y = y / torch.sqrt(y.square().sum(-1, keepdim=True) / d + 1e-6) * w.double()
        z = torch.complex(y[..., first], y[..., second]) * turn[:, None, :]
        out = y.clone()
        out[..., first], out[..., second] = z.real, z.imag
        return out

    def store(pool, x, scale):
        if c["fp8"]:
            old = pool.view(torch.float8_e4m3fn).double()
            x = (x / scale).clamp(-448.0, 448.0)
        else:
            old = pool.double()
        old.index_copy_(0, s["slots"].long(), x)
        return old

    return {"q": rows(s["q"], s["qw"]),
            "pool_k": store(s["pool_k"], rows(s["k"], s["kw"]), s.get("k_scale")),
            "pool_v": store(s["pool_v"], s["v"].double(), s.get("v_scale"))}


def _exact_attention(s):
    c = s["case"]
    hq, hkv, d, g = c["hq"], c["hkv"], c["d"], c["hq"] // c["hkv"]
    out = torch.empty(s["q"].shape, dtype=torch.float64, device=DEV)
    table, rpi = s["req_to_token"].cpu(), s["req_pool_idx"].tolist()
    value = {}
    for w in ("k", "v"):
        value[w] = ((lambda i, w=w: s["pool_" + w][i].view(torch.float8_e4m3fn).double() * s[w + "_scale"])
                    if c["fp8"] else (lambda i, w=w: s["pool_" + w][i].double()))
    at = 0
    for r in range(c["b"]):
        p, e = s["prefix"][r], s["ext"][r]
        for t0 in range(0, e, 256):
            t1 = min(e, t0 + 256)
            # every position the last query of the block may see, masked query by query
            keep = [j for j in range(p + t1) if j < c["sinks"] or j > p + t0 - c["window"]]
            pos = torch.tensor(keep, device=DEV)
            idx = table[rpi[r], keep].long().to(DEV)
            k, v = value["k"](idx), value["v"](idx)
            away = p + torch.arange(t0, t1, device=DEV)[:, None] - pos
            hidden = (away < 0) | ((away >= c["window"]) & (pos >= c["sinks"]))
            for h in range(hkv):
                q = s["q"][at + t0: at + t1, h * g: (h + 1) * g].double()
                score = torch.einsum("tgd,jd->tgj", q, k[:, h]) * d ** -0.5
                score[hidden[:, None].expand_as(score)] = -math.inf
                prob = torch.softmax(score, -1)
                out[at + t0: at + t1, h * g: (h + 1) * g] = torch.einsum("tgj,jd->tgd", prob, v[:, h])
        at += e
    return out
