"""Cases of a speculative decoding step: what a serving loop calls once a draft
model has proposed a tree of tokens for each running request.

  verify  attention of the drafted tokens: each sees its request's cached prefix
          and its own ancestors; a prefix that the whole batch shares is read once
  accept  the walk down each tree against the target's probabilities, from given
          random numbers, and the token drawn where it ends
  commit  the accepted tokens' slots enter req_to_token, the others' are freed

Each case is a dict of plain values; ``prepare`` makes its inputs on the GPU,
``run`` makes one pass (the framework's call where ``own`` is true, elementary
torch operations elsewhere) and ``exact`` computes the same outputs from the
definition in 64 bits.
"""
import math
import random

import torch

own = False
DEV = "cuda"


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one interactive request far into its context, a chain of 4 drafts and the root
        dict(name="verify_single_16k", op="verify", b=1, pre_lo=16384, pre_hi=16384, n_lo=5, n_hi=5, tree=False,
             shared=0, hq=32, hkv=8, d=128, fp8=False, seed=1),
        # 64 requests of a few thousand tokens, trees of 16
        dict(name="verify_64_tree_16", op="verify", b=64, pre_lo=512, pre_hi=4096, n_lo=16, n_hi=16, tree=True,
             shared=0, hq=32, hkv=8, d=128, fp8=False, seed=2),
        # 128 long multi-turn requests, chains of 8
        dict(name="verify_128_long", op="verify", b=128, pre_lo=1024, pre_hi=32768, n_lo=8, n_hi=8, tree=False,
             shared=0, hq=16, hkv=8, d=128, fp8=False, seed=3),
        # an e4m3 pool, ragged trees of up to 32
        dict(name="verify_48_fp8", op="verify", b=48, pre_lo=1000, pre_hi=16000, n_lo=3, n_hi=32, tree=True,
             shared=0, hq=32, hkv=8, d=128, fp8=True, seed=4),
        # heads of 64, three query heads a KV head, trees of up to 64 that fill several tiles
        dict(name="verify_33_d64", op="verify", b=33, pre_lo=0, pre_hi=2500, n_lo=1, n_hi=64, tree=True,
             shared=0, hq=12, hkv=4, d=64, fp8=False, seed=5),
        # 64 requests behind one 4,096-token system prompt
        dict(name="verify_shared_4096", op="verify", b=64, pre_lo=4100, pre_hi=4600, n_lo=8, n_hi=8, tree=True,
             shared=4096, hq=32, hkv=8, d=128, fp8=False, seed=6),
        # one request, a chain of drafts picked greedily
        dict(name="accept_single_chain", op="accept", b=1, n_lo=5, n_hi=5, tree=False, probs=False, vocab=32000,
             seed=7),
        # 64 requests, chains drawn from the draft model's distribution
        dict(name="accept_64_chain", op="accept", b=64, n_lo=6, n_hi=6, tree=False, probs=True, vocab=131072, seed=8),
        # ragged trees drawn from the draft model, a vocabulary that no vector width divides
        dict(name="accept_24_tree", op="accept", b=24, n_lo=2, n_hi=24, tree=True, probs=True, vocab=50257, seed=9),
        # a large batch of trees of the draft model's most likely tokens
        dict(name="accept_200_tree", op="accept", b=200, n_lo=1, n_hi=8, tree=True, probs=False, vocab=131072,
             seed=10),
        # slots of one request's tree
        dict(name="commit_1", op="commit", b=1, n_lo=5, n_hi=5, tree=False, seed=11),
        # slots of a large batch of ragged trees
        dict(name="commit_512", op="commit", b=512, n_lo=0, n_hi=64, tree=True, seed=12),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["verify", "verify", "verify", "accept", "accept", "commit"])
    n_hi = _log_int(rng, 1, 64)
    c = dict(op=op, n_hi=n_hi, n_lo=rng.choice([1, n_hi, max(1, n_hi // 3)]), tree=rng.random() < 0.6,
             seed=rng.randrange(1 << 30))
    if op == "commit":
        return dict(c, b=_log_int(rng, 1, 512))
    if op == "accept":
        vocab = _log_int(rng, 1000, 131072)
        return dict(c, b=max(1, min(_log_int(rng, 1, 200), (1 << 27) // (n_hi * vocab))), vocab=vocab,
                    probs=rng.random() < 0.6)
    d = rng.choice([64, 128, 128])
    hkv = rng.choice([1, 2, 3, 4, 8, 8])
    g = rng.choice([1, 2, 2, 3, 4, 4, 5, 8])
    pre = _log_int(rng, 1, 32768)
    shared = pre // rng.choice([1, 2, 4]) if rng.random() < 0.25 else 0
    b = max(1, min(_log_int(rng, 1, 160), 400000 // (pre + 1)))
    return dict(c, b=b, pre_lo=max(shared, pre // rng.choice([1, 3, 32])), pre_hi=pre, shared=shared, hq=hkv * g,
                hkv=hkv, d=d, fp8=rng.random() < 0.4)


def _lens(case):
    """Drafted tokens of each request, and its prefix."""
    rng = random.Random(case["seed"])
    n = [rng.randint(case["n_lo"], case["n_hi"]) for _ in range(case["b"])]
    pre = []
    if case["op"] == "verify":
        lo, hi = case["pre_lo"], case["pre_hi"]
        pre = [_log_int(rng, lo, hi) if lo > 0 and hi >= 16 * lo else rng.randint(lo, hi) for _ in range(case["b"])]
    return n, pre


def _parents(case, n):
    """Each node's parent among its request's nodes: node 0, the root, has none."""
    rng = random.Random(case["seed"] + 1)
    pick = (lambda i: rng.randint(max(0, i - 5), i - 1)) if case["tree"] else (lambda i: i - 1)
    return [[-1 if i == 0 else pick(i) for i in range(x)] for x in n]


def _ancestors(par):
    """The node and its ancestors, node by node."""
    seen = []
    for i, p in enumerate(par):
        seen.append((seen[p] if p >= 0 else []) + [i])
    return seen


def work(case):
    n, pre = _lens(case)
    tokens, b = sum(n), case["b"]
    if case["op"] == "commit":
        # lengths, counts and paths in; slots in and out; new lengths out
        return {"bytes": 4 * (6 * b + 3 * tokens), "flops": tokens}
    if case["op"] == "accept":
        rows = b * case["vocab"] * (2 if case["probs"] else 1)
        return {"bytes": 4 * (rows + 3 * tokens + 4 * b + b * max(n)), "flops": rows}
    hq, hkv, d, shared = case["hq"], case["hkv"], case["d"], case["shared"]
    own_pairs = sum(len(s) for par in _parents(case, n) for s in _ancestors(par))
    pairs = own_pairs + sum(x * p for x, p in zip(n, pre))
    keys = shared + sum(p + x - shared for x, p in zip(n, pre) if x)
    return {"bytes": keys * (2 * hkv * d * (1 if case["fp8"] else 2) + 4) + tokens * (4 * hq * d + 4),
            "flops": 4 * d * hq * pairs}


# ------------------------------------------------------------------ inputs

def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device=DEV, dtype=torch.bfloat16)


def _codes(x, scale):
    """e4m3 codes of bf16 rows, saturating."""
    return (x.float() / scale).clamp_(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    n, pre = _lens(case)
    par = _parents(case, n)
    s = dict(case=case, n=n, pre=pre, par=par, total=sum(n), most=max(1, max(n)))
    s["draft_lens"] = _ints(n)
    s["parents"] = _ints([p for row in par for p in row])
    {"verify": _prepare_verify, "accept": _prepare_accept, "commit": _prepare_commit}[case["op"]](s, gen)
    return s


def _prepare_verify(s, gen):
    c, n, pre = s["case"], s["n"], s["pre"]
    hq, hkv, d, b, shared = c["hq"], c["hkv"], c["d"], c["b"], c["shared"]
    live = shared + sum(p + x - shared for p, x in zip(pre, n))
    pool = live + live // 8 + 64
    perm = torch.randperm(pool, generator=gen, device=DEV).to(torch.int32)
    rows, stride = b + 3, max(p + x for p, x in zip(pre, n)) + 5
    s["req_to_token"] = torch.randint(0, pool, (rows, stride), generator=gen, device=DEV, dtype=torch.int32)
    rpi = list(range(rows))
    random.Random(c["seed"]).shuffle(rpi)
    s["rows"], s["req_pool_idx"] = rpi[:b], _ints(rpi[:b])
    at = shared
    for r, (p, x) in enumerate(zip(pre, n)):
        row = s["req_to_token"][rpi[r]]
        row[:shared] = perm[:shared]
        row[shared: p + x] = perm[at: at + p + x - shared]
        at += p + x - shared
    s["pool_k"], s["pool_v"] = _randn(gen, pool, hkv, d), _randn(gen, pool, hkv, d)
    # a request's first token draws a good part of every query's weight
    lead = _randn(gen, hkv, 1, d)
    first = s["req_to_token"][s["req_pool_idx"].long(), 0].long().unique()
    s["pool_k"][first] += (0.9 * lead[:, 0]).to(torch.bfloat16)
    if c["fp8"]:
        s["k_scale"], s["v_scale"] = 0.02, 0.0173
        s["pool_k"], s["pool_v"] = _codes(s["pool_k"], s["k_scale"]), _codes(s["pool_v"], s["v_scale"])
    s["q"] = (_randn(gen, s["total"], hkv, hq // hkv, d) + 0.7 * lead).reshape(s["total"], hq, d).contiguous()
    s["out"] = torch.empty_like(s["q"])
    s["prefix_lens"] = _ints(pre)
    if own:
        from radixattention_prefix_shared_gb300 import binding as B
        s["workspace"] = B.new_workspace(B.verify_workspace_bytes(b, s["total"], s["most"], max(pre), shared,
                                                                  B.make_dims(hq, hkv, d, pool)), DEV)


def _ranks(par):
    """Each node's place among its siblings."""
    met = {}
    ranks = []
    for p in par:
        ranks.append(met.get(p, 0))
        met[p] = ranks[-1] + 1
    return ranks


def _prepare_accept(s, gen):
    c, n, vocab = s["case"], s["n"], s["case"]["vocab"]
    # two models that mostly agree
    base = torch.randn(s["total"], vocab, generator=gen, device=DEV) * 3.5
    s["target_probs"] = torch.softmax(base, -1)
    base += torch.randn(s["total"], vocab, generator=gen, device=DEV)
    q = torch.softmax(base, -1)
    del base
    starts = [sum(n[:r]) for r in range(len(n))]
    above = torch.tensor([a + max(p, 0) for a, par in zip(starts, s["par"]) for p in par], device=DEV)
    if c["probs"]:
        # drawn from the draft model's distribution at the parent
        tokens = torch.multinomial(q[above], 1, generator=gen)[:, 0]
    else:
        # its most likely tokens at the parent
        rank = torch.tensor([k for par in s["par"] for k in _ranks(par)], device=DEV)
        tokens = torch.topk(q, min(vocab, s["most"])).indices[above, rank]
    s["draft_tokens"] = tokens.to(torch.int32)
    s["draft_probs"] = q if c["probs"] else None
    s["coins"] = torch.rand(s["total"], generator=gen, device=DEV)
    s["final_coins"] = torch.rand(c["b"], generator=gen, device=DEV)


def _prepare_commit(s, gen):
    c, n, b = s["case"], s["n"], s["case"]["b"]
    rng = random.Random(c["seed"] + 2)
    lens = [rng.randint(1, 4000) for _ in range(b)]
    paths = []
    for par in s["par"]:
        # a path from the root to some node
        paths.append(_ancestors(par)[rng.randrange(len(par))] if par else [])
    s["lens"], s["paths"] = lens, paths
    s["prefix_lens"] = _ints(lens)
    s["accepted"] = _ints([p + [-1] * (s["most"] - len(p)) for p in paths])
    s["num_accepted"] = _ints([len(p) for p in paths])
    pool = 4 * s["total"] + 64
    s["slots"] = torch.randperm(pool, generator=gen, device=DEV)[: s["total"]].to(torch.int32)
    s["req_to_token"] = torch.randint(0, pool, (b + 3, 4000 + s["most"] + 5), generator=gen, device=DEV,
                                      dtype=torch.int32)
    rpi = list(range(b + 3))
    rng.shuffle(rpi)
    s["rows"], s["req_pool_idx"] = rpi[:b], _ints(rpi[:b])
    s["seq_lens"] = torch.empty(b, dtype=torch.int32, device=DEV)
    # freed slots are listed from the front; what lies behind them stays as it was
    s["freed"] = torch.full((s["total"],), -1, dtype=torch.int32, device=DEV)
    s["num_freed"] = torch.empty(1, dtype=torch.int32, device=DEV)


# ------------------------------------------------------------------ one pass

def run(s):
    op = s["case"]["op"]
    if own:
        return {"verify": _own_verify, "accept": _own_accept, "commit": _own_commit}[op](s)
    return {"verify": _plain_verify, "accept": _plain_accept, "commit": _plain_commit}[op](s)


def _own_verify(s):
    from radixattention_prefix_shared_gb300 import binding as B
    c = s["case"]
    kw = dict(out=s["out"], max_draft=s["most"], max_prefix=max(s["pre"]), shared_len=c["shared"],
              workspace=s["workspace"])
    if c["fp8"]:
        return B.sgl_verify_attention_fp8(s["q"], s["pool_k"], s["pool_v"], s["k_scale"], s["v_scale"],
                                          s["req_to_token"], s["req_pool_idx"], s["prefix_lens"], s["draft_lens"],
                                          s["parents"], **kw)
    return B.sgl_verify_attention(s["q"], s["pool_k"], s["pool_v"], s["req_to_token"], s["req_pool_idx"],
                                  s["prefix_lens"], s["draft_lens"], s["parents"], **kw)


def _own_accept(s):
    from radixattention_prefix_shared_gb300 import binding as B
    path, count, token = B.sgl_verify_drafts(s["target_probs"], s["draft_tokens"], s["parents"], s["draft_lens"],
                                             s["coins"], s["final_coins"], s["draft_probs"], max_draft=s["most"])
    return {"accepted": path, "num_accepted": count, "next_tokens": token}


def _own_commit(s):
    from radixattention_prefix_shared_gb300 import binding as B
    B.sgl_commit_drafts(s["req_to_token"], s["req_pool_idx"], s["prefix_lens"], s["draft_lens"], s["slots"],
                        s["accepted"], s["num_accepted"], seq_lens=s["seq_lens"], freed=s["freed"],
                        num_freed=s["num_freed"])
    return {k: s[k] for k in ("req_to_token", "seq_lens", "freed", "num_freed")}


# ------------------------------------------------------------------ plain forms

def _plain_verify(s):
    c, par, n = s["case"], s["parents"].long(), s["n"]
    hkv, d = c["hkv"], c["d"]
    # sees[t, i]: node i of t's request is t or above it; each step goes one parent up
    node = torch.cat([torch.arange(x, device=DEV) for x in n])
    sees = torch.zeros(s["total"], s["most"], dtype=torch.bool, device=DEV)
    start = torch.arange(s["total"], device=DEV) - node
    at = node.clone()
    for _ in range(s["most"]):
        sees.scatter_(1, at[:, None], True)
        up = par[start + at]
        at = torch.where(up >= 0, up, at)
    t0 = 0
    for r, (p, x) in enumerate(zip(s["pre"], n)):
        slots = s["req_to_token"][s["rows"][r], : p + x].long()
        k, v = s["pool_k"][slots], s["pool_v"][slots]
        if c["fp8"]:
            k = k.view(torch.float8_e4m3fn).float() * s["k_scale"]
            v = v.view(torch.float8_e4m3fn).float() * s["v_scale"]
        k, v = k.float().transpose(0, 1)[:, None], v.float().transpose(0, 1)[:, None]
        q = s["q"][t0: t0 + x].float().view(x, hkv, -1, d).permute(1, 2, 0, 3)
        sc = (q @ k.transpose(-1, -2)) / math.sqrt(d)
        sc[..., p:] = sc[..., p:].masked_fill(~sees[t0: t0 + x, :x], float("-inf"))
        w = torch.exp(sc - sc.amax(-1, keepdim=True))
        o = (w @ v) / w.sum(-1, keepdim=True)
        s["out"][t0: t0 + x] = o.permute(2, 0, 1, 3).reshape(x, -1, d).to(torch.bfloat16)
        t0 += x
    return s["out"]


def _plain_accept(s):
    # in 64 bits: residuals are differences of nearly equal values, and the
    # drawn token lies next to a border of a long sum
    b, vocab, most = s["case"]["b"], s["case"]["vocab"], s["most"]
    n = s["draft_lens"].long()
    start = torch.cumsum(n, 0) - n
    each = torch.arange(b, device=DEV)
    p, q = s["target_probs"], s["draft_probs"]
    here = torch.zeros(b, dtype=torch.long, device=DEV)   # the last accepted node
    left, mass = p[start].double(), torch.ones(b, dtype=torch.float64, device=DEV)
    path = torch.full((b, most), -1, dtype=torch.int32, device=DEV)
    path[:, 0] = 0
    count = torch.ones(b, dtype=torch.long, device=DEV)
    for i in range(1, most):
        t = torch.clamp(start + i, max=s["total"] - 1)
        asked = (i < n) & (s["parents"][t] == here)
        token = s["draft_tokens"][t].long()
        weight = left[each, token]
        drawn = q[start + here, token].double() if q is not None else 1.0
        taken = asked & (weight > 0) & (s["coins"][t].double() * drawn * mass < weight)
        path[each, torch.clamp(count, max=most - 1)] = torch.where(
            taken, i, path[each, torch.clamp(count, max=most - 1)]).to(torch.int32)
        count += taken
        lost = asked & ~taken
        if q is not None:
            rest = torch.clamp(left / mass[:, None] - q[start + here].double(), min=0)
            sums = rest.sum(-1)
        else:
            rest = left.index_put((each, token), torch.zeros((), dtype=torch.float64, device=DEV))
            sums = mass - weight
        here = torch.where(taken, i, here)
        left = torch.where(taken[:, None], p[start + here].double(), torch.where(lost[:, None], rest, left))
        mass = torch.where(taken, 1.0, torch.where(lost, sums, mass))
    left = torch.where(left.sum(-1, keepdim=True) > 0, left, p[start + here].double())
    cum = torch.cumsum(left, -1)
    token = (cum > s["final_coins"].double()[:, None] * cum[:, -1:]).long().argmax(-1)
    return {"accepted": path, "num_accepted": count.to(torch.int32), "next_tokens": token.to(torch.int32)}


def _plain_commit(s):
    n, count = s["draft_lens"].long(), s["num_accepted"].long()
    start = torch.cumsum(n, 0) - n
    k = torch.arange(s["most"], device=DEV)[None]
    kept = k < count[:, None]
    req, at = kept.nonzero(as_tuple=True)
    token = start[req] + s["accepted"][req, at].long()
    s["req_to_token"][s["req_pool_idx"].long()[req], s["prefix_lens"].long()[req] + at] = s["slots"][token]
    s["seq_lens"].copy_(s["prefix_lens"] + s["num_accepted"])
    free = torch.ones(s["total"], dtype=torch.bool, device=DEV)
    free[token] = False
    out = s["slots"][free]
    s["freed"][: out.numel()] = out
    s["num_freed"].fill_(out.numel())
    return {k: s[k] for k in ("req_to_token", "seq_lens", "freed", "num_freed")}


# ------------------------------------------------------------------ 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "verify":
        return _exact_verify(s)
    return None   # tokens, slots and lengths are whole numbers


def _exact_verify(s):
    c = s["case"]
    hkv, g, d = c["hkv"], c["hq"] // c["hkv"], c["d"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    table = s["req_to_token"].cpu()
    t0 = 0
    for r, (p, par) in enumerate(zip(s["pre"], s["par"])):
        x = len(par)
        hidden = torch.ones(x, x, dtype=torch.bool)
        for i, seen in enumerate(_ancestors(par)):
            hidden[i, seen] = False
        hidden = torch.cat((torch.zeros(x, p, dtype=torch.bool), hidden), 1).to(DEV)
        idx = table[s["rows"][r], : p + x].long().to(DEV)
        for h in range(hkv):
            k, v = s["pool_k"][idx, h], s["pool_v"][idx, h]
            if c["fp8"]:
                k = k.view(torch.float8_e4m3fn).double() * s["k_scale"]
                v = v.view(torch.float8_e4m3fn).double() * s["v_scale"]
            for e in range(h * g, (h + 1) * g):
                score = s["q"][t0: t0 + x, e].double() @ k.double().T * d ** -0.5
                score[hidden] = -math.inf
                out[t0: t0 + x, e] = torch.softmax(score, -1) @ v.double()
        t0 += x
    return out
