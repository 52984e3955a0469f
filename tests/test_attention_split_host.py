"""The sums that the attention's split of the work rests on, run on the host:
units of a sequence's row tiles (key tiles that any of its rows sees, at least
one, and a weight each), against the same in Python's integers."""

import subprocess

import pytest

from all_reduce_reduction_rank_gb300 import build as arbuild

CASES = [(1, 1, 1, 0), (1, 64, 8, 0), (1, 65, 8, 0), (3, 2, 2, 0), (5, 0, 16, 0), (300, 300, 4, 0), (300, 1000, 4, 100),
         (513, 640, 7, 1), (9, 4, 16, 1 << 30), (4096, 131072, 1, 0),
         # more than 2^32 units in one sequence
         (1_000_000, 1_000_000, 1, 0), (600_000, 1_500_000, 1, 0), (1_000_000, 900_000, 1, 0)]


def units(nq, kv, tm, window, keys, weight):
    total = 0
    for t in range(0, nq, tm):
        first = kv - nq + t
        hi = max(kv - nq + min(t + tm, nq), 0)
        lo = max(first - window + 1, 0) if window else 0
        total += max(-(-hi // keys) - lo // keys, 1) + weight
    return total


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    exe = tmp_path_factory.mktemp("split") / "split_host"
    src = arbuild.ROOT / "tests" / "split_host.cu"
    subprocess.run([arbuild.nvcc(), *arbuild.ARCH, "-std=c++17", "-I", str(arbuild.INCLUDE), "-I", str(arbuild.CSRC),
                    str(src), "-o", str(exe)], check=True)
    return exe


def test_units_of_a_sequence(program):
    text = "".join("%d %d %d %d\n" % c for c in CASES)
    got = subprocess.run([str(program)], input=text, capture_output=True, text=True, check=True).stdout.split()
    want = [units(*c, keys, weight) for c in CASES for keys, weight in ((64, 1), (128, 3))]
    assert [int(x) for x in got] == want
    assert sum(w > 2**32 for w in want) >= 3
