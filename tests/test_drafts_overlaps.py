"""Buffers of the drafted-token calls that overlap: refused on the host (no call here
gets as far as a launch)."""
import ctypes

import pytest

INVALID = 1
T, BATCH, MOST, V = 12, 3, 6, 100
ROWS, STRIDE = 4, 40

WALK_IN = dict(p=4 * (T - 1) * 120 + 4 * V, q=4 * (T - 1) * 130 + 4 * V, tok=4 * T, par=4 * T, dl=4 * BATCH,
               coins=4 * T, final=4 * BATCH)
WALK_OUT = dict(acc=4 * BATCH * MOST, num=4 * BATCH, nxt=4 * BATCH)


def _apart(names):
    """An address for each buffer, far from the others'."""
    return {n: 0x10000000 * (i + 1) for i, n in enumerate(names)}


def _ptr(x):
    return None if x is None else ctypes.c_void_p(x)


def walk(lib, at):
    return lib.sgl_verify_drafts(_ptr(at["p"]), 120, _ptr(at["q"]), 130, V, _ptr(at["tok"]), _ptr(at["par"]),
                                 _ptr(at["dl"]), BATCH, T, MOST, _ptr(at["coins"]), _ptr(at["final"]), _ptr(at["acc"]),
                                 _ptr(at["num"]), _ptr(at["nxt"]), None)


@pytest.mark.parametrize("out", WALK_OUT)
@pytest.mark.parametrize("other", [*WALK_IN, *WALK_OUT])
def test_walk(cuda_lib, out, other):
    if out == other:
        return
    sizes = WALK_IN | WALK_OUT
    at = _apart(sizes)
    for where in (at[other], at[other] + sizes[other] - 4, at[other] - sizes[out] + 4):
        assert walk(cuda_lib, at | {out: where}) == INVALID
