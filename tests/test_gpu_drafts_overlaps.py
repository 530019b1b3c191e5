"""Drafted-token calls whose buffers overlap are refused before they launch; buffers that
only touch are not."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import oracle  # noqa: E402
from radixattention_prefix_shared_gb300 import binding as B  # noqa: E402

from _drafts import accept_case, want_accept  # noqa: E402
from test_gpu_drafts import commit_case  # noqa: E402

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]

DEV = "cuda:0"


def _refused(f, *args, **kw):
    with pytest.raises(B.SglError) as e:
        f(*args, **kw)
    assert e.value.code == 1


def test_walk():
    c = accept_case(301, drafts=[5, 0, 3, 6], V=700)
    up = lambda x: torch.from_numpy(x).to(DEV)  # noqa: E731
    tok, par, lens, final = up(c["tok"]), up(c["parents"]), up(c["drafts"]), up(c["final"])
    most, T = c["most"], len(c["tok"])
    args = [up(c["p"]), tok, par, lens, up(c["coins"]), final, up(c["q"])]
    for kw in (dict(num_accepted=lens), dict(next_tokens=lens), dict(next_tokens=tok[1:5]), dict(num_accepted=par[-4:]),
               dict(next_tokens=final.view(torch.int32)), dict(accepted=args[0].view(torch.int32).view(-1)[: 4 * most].view(4, most)),
               dict(accepted=args[6].view(torch.int32).view(-1)[-4 * most:].view(4, most))):
        _refused(B.sgl_verify_drafts, *args, max_draft=most, **kw)
    one = torch.zeros(4 * most + 8, dtype=torch.int32, device=DEV)
    _refused(B.sgl_verify_drafts, *args, max_draft=most, num_accepted=one[:4], next_tokens=one[3:7])
    # one buffer for all that is small: neighbours that only touch
    flat = torch.cat([tok, par, lens, one])
    tok2, par2, lens2 = flat[:T], flat[T: 2 * T], flat[2 * T: 2 * T + 4]
    rest = flat[2 * T + 4:]
    got = B.sgl_verify_drafts(args[0], tok2, par2, lens2, args[4], final, args[6], max_draft=most,
                              accepted=rest[4:-4].view(4, most), num_accepted=rest[:4], next_tokens=rest[-4:])
    for x, w in zip(got, want_accept(c)):
        assert np.array_equal(x.cpu().numpy(), w)


def test_commit():
    c = commit_case(302, [3, 0, 7, 20, 1])
    new = lambda: [torch.from_numpy(c[k]).to(DEV) for k in ("rtt", "rpi", "pre", "drafts", "slots", "acc", "cnt")]  # noqa: E731
    t = new()
    rtt, rpi, pre, lens, slots, acc, cnt = t
    for kw in (dict(freed=slots), dict(seq_lens=cnt), dict(seq_lens=lens), dict(seq_lens=rpi), dict(seq_lens=slots[2:7]),
               dict(num_freed=pre[:1]), dict(num_freed=rtt.view(-1)[5:6]), dict(freed=acc.view(-1)[: len(slots)])):
        _refused(B.sgl_commit_drafts, *t, **kw)
    # the one request's slots as they stand in its row
    view = rtt.view(-1)[5: 5 + len(slots)]
    _refused(B.sgl_commit_drafts, *t[:4], view, acc, cnt)
    assert all(torch.equal(a, b) for a, b in zip(t, new()))
    # the new lengths in place of the old ones, over many requests
    c = commit_case(303, [7] * 200)
    rtt, rpi, pre, lens, slots, acc, cnt = t = new()
    seq, freed, count = B.sgl_commit_drafts(*t, seq_lens=pre)
    want = oracle.drafts.commit_drafts(c["rtt"], c["rpi"], c["pre"], c["drafts"], c["slots"], c["acc"], c["cnt"])
    assert seq.data_ptr() == pre.data_ptr() and np.array_equal(seq.cpu().numpy(), want[1])
    assert np.array_equal(rtt.cpu().numpy(), want[0]) and np.array_equal(freed.cpu().numpy()[: len(want[2])], want[2])
    assert count.tolist() == [len(want[2])]
