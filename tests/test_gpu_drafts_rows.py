"""The walk over rows as a server cuts them: a few weights (top-k, top-p), one weight
(greedy), and large vocabularies, against the fp64 oracle, exactly."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from _drafts import accept_case  # noqa: E402
from test_gpu_drafts import check_accept  # noqa: E402

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]


def _cut(rows, k):
    """A row's k largest weights, scaled to sum to 1."""
    out = np.zeros_like(rows)
    at = np.argpartition(-rows, k - 1, axis=-1)[:, :k]
    top = np.take_along_axis(rows, at, -1).astype(np.float64)
    np.put_along_axis(out, at, (top / top.sum(-1, keepdims=True)).astype(np.float32), -1)
    return out


def _redraw(c, g):
    """Tokens drawn anew from the draft rows of their parents."""
    starts = np.repeat(np.cumsum(np.append(0, c["drafts"]))[:-1], c["drafts"])
    for t, s in enumerate(starts):
        row = c["q"][s + max(0, c["parents"][t])].astype(np.float64)
        c["tok"][t] = g.choice(c["V"], p=row / row.sum())


@pytest.mark.parametrize("drawn", [True, False])
@pytest.mark.parametrize("kind", ["chain", "tree", "bush"])
@pytest.mark.parametrize("V,k", [(40, 1), (40, 3), (5003, 1), (5003, 8), (5003, 50), (50257, 20)])
def test_rows_of_a_few_weights(V, k, kind, drawn):
    g = np.random.default_rng(V + k)
    c = accept_case(700 + k, drafts=[1, 8, 3, 24, 5], V=V, kind=kind, drawn=drawn)
    c["p"] = _cut(c["p"], k)
    if drawn:
        c["q"] = _cut(c["q"], min(V, 2 * k))
        _redraw(c, g)
    else:   # half of the drafts are the target's own choice at the parent
        starts = np.repeat(np.cumsum(np.append(0, c["drafts"]))[:-1], c["drafts"])
        best = c["p"].argmax(-1)[starts + np.maximum(c["parents"], 0)]
        c["tok"] = np.where(g.random(c["tok"].size) < 0.5, best, c["tok"]).astype(np.int32)
    check_accept(c)


@pytest.mark.parametrize("drawn", [True, False])
def test_the_same_rows_in_both_models(drawn):
    """A draft model that is the target: its draws are rejected by a coin of 1 alone."""
    c = accept_case(720, drafts=[9, 9, 9], V=3001, drawn=True)
    c["p"] = c["q"].copy()
    c["coins"][9 + 4] = 1.0
    if not drawn:
        c["q"] = None
    check_accept(c)


@pytest.mark.parametrize("drawn", [True, False])
@pytest.mark.parametrize("V", [131072, 200003, 262144])
def test_large_vocabularies(V, drawn):
    check_accept(accept_case(730, drafts=[7, 1, 12], V=V, kind="tree", drawn=drawn))
    check_accept(accept_case(731, drafts=[2] * 40, V=V, kind="chain", drawn=drawn))
    check_accept(accept_case(732, drafts=[20], V=V, kind="bush", drawn=drawn))
    c = accept_case(733, drafts=[5, 5], V=V, drawn=drawn)
    c["p"] = _cut(c["p"], 40)
    check_accept(c)
