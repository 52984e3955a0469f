"""The sums that the scored attention's split of the work rests on, run on the
host: units of a sequence's row tiles where prefixes show keys behind a row and
documents hide keys before it, against the same in Python's integers."""

import random
import subprocess

import pytest

from all_reduce_reduction_rank_gb300 import build as arbuild

KINDS = ((64, 1), (128, 3), (128, 4))


def units(nq, kv, tm, window, prefix, first, keys, weight):
    """From what each row sees: its keys are [lo, hi), a row tile's from its first row's lo to its last one's hi."""
    total = 0
    for t in range(0, nq, tm):
        p, last = kv - nq + t, kv - nq + min(t + tm, nq) - 1
        hi = max(last + 1, min(prefix, kv)) if last >= 0 else 0
        lo = max(p - window + 1 if window else 0, first[t] if first else 0, 0)
        lo = min(lo, hi)
        total += max(-(-hi // keys) - lo // keys, 1) + weight
    return total


def cases():
    rng = random.Random(5)
    yield 1, 1, 1, 0, 0, None
    yield 5, 0, 2, 0, 9, None                              # no keys
    yield 7, 3, 2, 0, 3, None                              # positions before the first
    yield 3, 1000, 2, 0, 2**31 - 1, [0, 999, 2**31 - 1]    # a prefix and a document past the keys
    yield 3, 1000, 2, 5, -2**31, [-2**31, -1, 0]
    yield 1_000_000, 1_000_000, 1, 0, 900_000, None        # more than 2^32 units
    for _ in range(200):
        nq = rng.randint(1, 600)
        kv = max(0, nq + rng.randint(-5, 3000))
        first = sorted(rng.randint(-3, kv + 3) for _ in range(nq)) if rng.random() < 0.6 else None
        yield nq, kv, rng.choice([1, 2, 4, 8, 16, 32, 128]), rng.choice([0, 0, 1, 100, 1 << 30]), rng.randint(-2, kv + 2), first


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    exe = tmp_path_factory.mktemp("split") / "split_masked_host"
    src = arbuild.ROOT / "tests" / "split_masked_host.cu"
    subprocess.run([arbuild.nvcc(), *arbuild.ARCH, "-std=c++17", "-I", str(arbuild.INCLUDE), "-I", str(arbuild.CSRC),
                    str(src), "-o", str(exe)], check=True)
    return exe


def test_units_of_a_masked_sequence(program):
    todo = list(cases())
    text = "".join("%d %d %d %d %d %d %s\n" % (*c[:5], int(c[5] is not None), " ".join(map(str, c[5] or []))) for c in todo)
    got = subprocess.run([str(program)], input=text, capture_output=True, text=True, check=True).stdout.split()
    want = [units(*c, *kind) for c in todo for kind in KINDS]
    assert [int(x) for x in got] == want
    assert max(want) > 2**32
