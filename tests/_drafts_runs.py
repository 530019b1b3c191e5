"""Drafted-token batches large enough that a CTA takes several blocks of keys: how
the attention deals its blocks to CTAs, inputs made where they are used, and the
definition in float64 by matrix products (``oracle.drafts`` loops over rows)."""
from __future__ import annotations

import math

import numpy as np
import torch

from radixattention_prefix_shared_gb300 import binding as B

from _drafts import tree

BLOCK = 128      # keys of a block
MOST_CTAS = 160  # of a launch
MOST_STAGES = 12  # K and V slots of a CTA's rings


def columns(rows, fp8):
    """Columns of a tile that holds so many query rows a KV head."""
    return next((n for n in (16, 32, 64) if rows <= n), 64 if fp8 else 128)


def segments(prefix, drafts, Hq, Hkv, fp8, sms):
    """The blocks that each CTA takes of a unit (KV head, request, tile of columns),
    as (unit's blocks, first block, blocks taken), CTA by CTA; nothing shared."""
    g = Hq // Hkv
    n = columns(max(drafts) * g, fp8)
    units = []
    for _ in range(Hkv):
        for p, x in zip(prefix, drafts):
            if x > 0:
                units += [-(-(p + x) // BLOCK)] * -(-x * g // n)
    total = sum(units)
    ctas = min(sms, MOST_CTAS, total)
    out, unit, b = [], 0, 0
    for c in range(ctas):
        left, mine = total * (c + 1) // ctas - total * c // ctas, []
        while left:
            take = min(left, units[unit] - b)
            mine.append((units[unit], b, take))
            left, b = left - take, b + take
            if b == units[unit]:
                unit, b = unit + 1, 0
        out.append(mine)
    return out


class Batch:
    """Requests of ``drafts[r]`` nodes after ``prefix[r]`` tokens on ``dev``.  Entries of
    req_to_token behind a request's nodes name pool rows that are NaN.

    step: None, or by how much (in units of the softmax's exponent) the scores of a
    block of keys lie above those of the block before.  shared: positions whose slots
    are the same in every row."""

    def __init__(self, seed, *, Hq, Hkv, D, prefix, drafts, fp8=False, kind="tree", std=1.0, step=None, shared=0,
                 dev="cuda:0"):
        g = np.random.default_rng(seed)
        gen = torch.Generator(device=dev).manual_seed(seed)
        randn = lambda *s: torch.randn(*s, generator=gen, device=dev)  # noqa: E731
        self.Hq, self.Hkv, self.D, self.fp8, self.shared = Hq, Hkv, D, fp8, shared
        self.prefix, self.drafts = [int(x) for x in prefix], [int(x) for x in drafts]
        self.par = [tree(g, x, kind) for x in self.drafts]
        live = sum(p + x for p, x in zip(prefix, drafts))
        S, rows, stride = live + 9, len(drafts) + 2, max(p + x for p, x in zip(prefix, drafts)) + 3
        perm = g.permutation(S).astype(np.int32)
        rtt = perm[live + g.integers(0, 9, size=(rows, stride))]
        rpi = g.permutation(rows)[: len(drafts)].astype(np.int32)
        depth = np.zeros(S, np.int64)  # a slot's block in its request
        at, self.slots = 0, []
        for r, (p, x) in enumerate(zip(prefix, drafts)):
            mine = perm[at: at + p + x].copy()
            mine[:shared] = perm[:shared]
            rtt[rpi[r], : p + x] = mine
            depth[mine] = np.arange(p + x) // BLOCK
            self.slots.append(torch.from_numpy(mine.astype(np.int64)).to(dev))
            at += p + x
        k, v = randn(S, Hkv, D) * std, randn(S, Hkv, D)
        q = randn(max(1, sum(drafts)), Hq, D) * std
        if step is not None:
            # queries lie along u, at least 10 of it; keys rise along it block by block
            u, lift = 1 / math.sqrt(D), 12.0
            q = 0.3 * q + lift * u
            top = torch.from_numpy(depth - depth.max() / 2).to(dev)[:, None, None].float()
            k = 0.3 * k + top * (step * math.sqrt(D) / 10.0) * u
        self.scales = (float(k.abs().max()) / 400, 4 / 400) if fp8 else ()
        pools = []
        for x, s in zip((k, v), self.scales or (1.0, 1.0)):
            x = (x / s).clamp_(-448, 448).to(torch.float8_e4m3fn) if fp8 else x.to(torch.bfloat16)
            bits = x.view(torch.uint8 if fp8 else torch.int16)
            bits[torch.from_numpy(perm[live:].astype(np.int64)).to(dev)] = 0x7F if fp8 else 0x7FFF
            pools.append(bits if fp8 else x)
        self.pool_k, self.pool_v = pools
        self.q = q.to(torch.bfloat16)
        ints = lambda x: torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).to(dev)  # noqa: E731
        self.rtt, self.rpi = ints(rtt), ints(rpi)
        self.prefix_lens, self.draft_lens = ints(prefix), ints(drafts)
        self.parents = ints([i for p in self.par for i in p] or [-1])

    def new_workspace(self):
        return B.new_workspace(B.verify_workspace_bytes(len(self.drafts), sum(self.drafts), max(self.drafts),
                                                        max(self.prefix), self.shared,
                                                        B.make_dims(self.Hq, self.Hkv, self.D, len(self.pool_k))),
                               self.q.device)

    def run(self, **kw):
        f = B.sgl_verify_attention_fp8 if self.fp8 else B.sgl_verify_attention
        return f(self.q, self.pool_k, self.pool_v, *self.scales, self.rtt, self.rpi, self.prefix_lens,
                 self.draft_lens, self.parents, max_draft=max(self.drafts), max_prefix=max(self.prefix),
                 shared_len=self.shared, **kw)

    def segments(self):
        sms = torch.cuda.get_device_properties(0).multi_processor_count
        return segments(self.prefix, self.drafts, self.Hq, self.Hkv, self.fp8, sms)

    def _values(self, pool, r, i):
        """[KV heads, keys, D] of request r."""
        x = pool[self.slots[r]]
        x = x.view(torch.float8_e4m3fn).double() * self.scales[i] if self.fp8 else x.double()
        return x.transpose(0, 1)

    def visible(self, r):
        """[nodes, keys] of request r."""
        p, par = self.prefix[r], self.par[r]
        tree = np.zeros((len(par), len(par)), bool)
        for i, up in enumerate(par):
            if up >= 0:
                tree[i] = tree[up]
            tree[i, i] = True
        return torch.from_numpy(np.concatenate([np.ones((len(par), p), bool), tree], 1)).to(self.q.device)

    def _scores(self, r, see):
        g, t0, x = self.Hq // self.Hkv, sum(self.drafts[:r]), self.drafts[r]
        q = self.q[t0: t0 + x].double().view(x, self.Hkv, g, self.D).transpose(0, 1)
        k = self._values(self.pool_k, r, 0)[:, None].transpose(-1, -2)
        hidden = ~see[None, :, None]
        s, reach = (q @ k) * self.D ** -0.5, (q.abs() @ k.abs()) * self.D ** -0.5
        return s.masked_fill(hidden, -math.inf), reach.masked_fill(hidden, 0.0)

    def scores(self, r, h):
        """[nodes, heads of KV head h, keys] in float64, hidden ones -inf, and the
        products' absolute sums."""
        return tuple(x[h] for x in self._scores(r, self.visible(r)))

    def want(self):
        """(out, terms) as ``oracle.drafts.verify_attention``."""
        shape = self.q.shape
        out, spread = (torch.zeros(shape, dtype=torch.float64, device=self.q.device) for _ in range(2))
        reach, floor = (torch.zeros(*shape[:2], 1, dtype=torch.float64, device=self.q.device) for _ in range(2))
        t0 = 0
        for r, x in enumerate(self.drafts):
            if x == 0:
                continue
            see = self.visible(r)
            s, a = self._scores(r, see)
            v = self._values(self.pool_v, r, 1)[:, None]
            w = torch.exp(s - s.amax(-1, keepdim=True))
            total = w.sum(-1, keepdim=True)
            rows = lambda y: y.transpose(0, 1).flatten(1, 2)  # noqa: E731
            at = slice(t0, t0 + x)
            out[at], spread[at] = rows((w @ v) / total), rows((w @ v.abs()) / total)
            reach[at] = rows(a.amax(-1, keepdim=True))
            most = torch.where(see, v.abs().amax(-1), 0.0).amax(-1)[:, :, None, None]  # [KV heads, nodes, 1, 1]
            floor[at] = rows(see.sum(-1)[:, None, None] * most / total)
            t0 += x
        return out, dict(spread=spread, reach=reach, floor=floor)

    def check(self, what=""):
        """The bound of ``_drafts.assert_attention`` for every value; twice the same bits."""
        ws = self.new_workspace()
        got = self.run(workspace=ws)
        again = self.run(workspace=ws)
        assert int(ws[:4].view(torch.int32).item()) == 0, f"{what}: a wait gave up"
        rows = sum(self.drafts)
        want, t = self.want()
        bound = (2.0 ** -8 * want.abs() + (2.0 ** -8 + 2.0 ** -12 + 2.0 ** -16 * t["reach"]) * t["spread"]
                 + 2.0 ** -32 * t["floor"] + 1e-30)
        x = got[:rows].double()
        assert bool(torch.isfinite(x).all()), f"{what}: non-finite output"
        ratio = float(((x - want[:rows]).abs() / bound[:rows]).max())
        assert ratio <= 1.0, f"{what}: error {ratio:.3g} of its bound"
        assert torch.equal(got.view(torch.int16), again.view(torch.int16)), f"{what}: other bits when run again"
