"""The helpers of the large drafted-token batches: their float64 form against the
oracle's, and how blocks are dealt."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import oracle  # noqa: E402
from radixattention_prefix_shared_gb300 import workloads as W  # noqa: E402

from _drafts_runs import Batch, columns, segments  # noqa: E402


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("step", [None, 9.0])
def test_matrix_form_is_the_oracles(fp8, step):
    b = Batch(3, Hq=6, Hkv=2, D=64, prefix=[0, 130, 257], drafts=[5, 3, 7], fp8=fp8, step=step, dev="cpu")
    bits = (lambda x: x.numpy()) if fp8 else W.bf16_bits
    read = [oracle.window.pool_reader(bits(p), s) for p, s in zip((b.pool_k, b.pool_v), b.scales or (None, None))]
    out, terms = oracle.drafts.verify_attention(W.bf16_bits(b.q), *read, b.rtt.numpy(), b.rpi.numpy(), b.prefix,
                                                b.drafts, b.parents.numpy(), 2)
    got, got_terms = b.want()
    assert np.allclose(got.numpy(), out, rtol=1e-9, atol=1e-12)
    for name in terms:
        assert np.allclose(got_terms[name].numpy(), terms[name], rtol=1e-9, atol=1e-12), name


def test_keys_rise_block_by_block():
    b = Batch(4, Hq=8, Hkv=2, D=128, prefix=[400, 513], drafts=[4, 9], step=25.0, dev="cpu")
    for r, p in enumerate(b.prefix):
        for h in range(2):
            s, _ = b.scores(r, h)
            tops = torch.stack([s[..., i: i + 128].amax(-1) for i in range(0, p, 128)])
            assert float((tops[1:] - tops[:-1]).min()) > 21


def test_blocks_are_dealt_in_order():
    assert [columns(n, False) for n in (1, 16, 17, 64, 65, 500)] == [16, 16, 32, 64, 128, 128]
    assert columns(500, True) == 64
    # two heads of (3 blocks, two tiles of 64 columns with a block each) over 4 CTAs
    runs = segments([300, 0], [16, 40], 4, 2, True, 4)
    assert sum(t for c in runs for _, _, t in c) == 2 * (3 + 2)
    assert [sum(t for _, _, t in c) for c in runs] == [2, 3, 2, 3]
    assert runs[0] == [(3, 0, 2)] and runs[1][0] == (3, 2, 1)
