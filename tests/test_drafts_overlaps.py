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


SLOTS_IN = dict(rpi=4 * BATCH, pre=4 * BATCH, dl=4 * BATCH, slots=4 * T, acc=4 * BATCH * MOST, num=4 * BATCH)
SLOTS_OUT = dict(rtt=4 * ROWS * STRIDE, seq=4 * BATCH, freed=4 * T, nf=4)


def commit(lib, at):
    return lib.sgl_commit_drafts(_ptr(at["rtt"]), ROWS, STRIDE, _ptr(at["rpi"]), _ptr(at["pre"]), _ptr(at["dl"]),
                                 _ptr(at["slots"]), _ptr(at["acc"]), _ptr(at["num"]), BATCH, T, MOST, _ptr(at["seq"]),
                                 _ptr(at["freed"]), _ptr(at["nf"]), None)


@pytest.mark.parametrize("out", SLOTS_OUT)
@pytest.mark.parametrize("other", [*SLOTS_IN, *SLOTS_OUT])
def test_commit(cuda_lib, out, other):
    if out == other:
        return
    sizes = SLOTS_IN | SLOTS_OUT
    at = _apart(sizes)
    for where in (at[other], at[other] + sizes[other] - 4, at[other] - sizes[out] + 4):
        if (out, other, where) == ("seq", "pre", at["pre"]):
            continue    # the new lengths in the old ones' place
        assert commit(cuda_lib, at | {out: where}) == INVALID
