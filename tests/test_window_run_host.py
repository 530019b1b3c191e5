"""Which positions a sliding-window decode reads: `window_run_host.cpp`, the
kernels' own arithmetic compiled with g++, against the mask written out."""
import os
import shutil
import subprocess

import numpy as np
import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "radixattention_prefix_shared_gb300", "csrc")
TOP = 2**31 - 1


def positions(sinks, window, max_seq, seq_len):
    """Positions below max_seq that the query at seq_len - 1 sees, ascending."""
    lo = max(0, seq_len - window)
    end = min(seq_len, max_seq)
    if end <= 100000:
        return [j for j in range(max(0, end)) if j < sinks or j >= lo]
    return list(range(min(sinks, lo))) + list(range(lo, end))


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("needs g++")
    exe = tmp_path_factory.mktemp("window_run") / "window_run_host"
    cmd = ["g++", "-std=c++17", "-O1", "-Wall", "-Wextra", "-Werror", "-I", CSRC,
           os.path.join(HERE, "window_run_host.cpp"), "-o", str(exe)]
    res = subprocess.run(cmd, capture_output=True, text=True)
    assert res.returncode == 0, res.stdout + res.stderr
    return str(exe)


def run(program, cases):
    """Each case against the mask; a case: (sinks, window, max_seq, n_splits, seq_len)."""
    lines, chunks = [], []
    for sinks, window, max_seq, n_splits, seq_len in cases:
        keys = min(max_seq, sinks + window)          # what the host sizes the runs by
        chunks.append(-(-keys // n_splits))
        lines.append(f"{sinks} {window} {max_seq} {n_splits} {chunks[-1]} {seq_len}")
    res = subprocess.run([program], input="\n".join(lines), capture_output=True, text=True, timeout=60)
    assert res.returncode == 0, res.stderr
    got = [[int(x) for x in line.split()] for line in res.stdout.splitlines()]
    assert len(got) == len(cases)
    for case, chunk, (n, ns, *pos) in zip(cases, chunks, got):
        sinks, window, max_seq, n_splits, seq_len = case
        want = positions(sinks, window, max_seq, seq_len)
        assert n == len(want), case
        assert pos == (want if n <= 400 else want[:200] + want[-200:]), case
        assert ns == -(-n // chunk) and ns <= n_splits, case


def test_lengths_above_the_host_maximum(program):
    """A query past max_seq_len still sees its own window only, cut there."""
    run(program, [(2, 20, 50, 1, 60), (2, 20, 50, 3, 60), (2, 100, 50, 1, 60), (0, 20, 50, 1, 60),
                  (2, 20, 50, 1, 70), (2, 20, 50, 1, 71), (0, 20, 50, 1, 70), (0, 20, 50, 2, 1000), (7, 1, 5, 1, 9),
                  (60, 3, 50, 1, 52), (60, 3, 50, 1, 5000), (4, 20, 50, 1, TOP), (TOP, TOP, 50, 1, TOP)])


def test_every_small_case(program):
    run(program, [(sinks, window, max_seq, n_splits, seq_len) for sinks in (0, 1, 3, 9) for window in (1, 2, 5, 12)
                  for max_seq in (1, 4, 8, 13) for n_splits in (1, 2) if min(max_seq, sinks + window) >= n_splits
                  for seq_len in range(-2, 16)])


def test_random_and_largest_values(program):
    g = np.random.default_rng(5)
    cases = []
    for _ in range(400):
        sinks, window, max_seq, seq_len = (int(np.exp(g.uniform(0, np.log(5000)))) for _ in range(4))
        cases.append((sinks - 1, window, max_seq, int(g.integers(1, 5)), seq_len))
    cases = [c for c in cases if min(c[2], c[0] + c[1]) >= c[3]]
    cases += [(4, 1000, TOP, 4, TOP), (TOP, 1000, 3000, 2, 2999), (0, TOP, 4096, 4, TOP), (3, 500, TOP, 2, TOP - 1)]
    run(program, cases)
