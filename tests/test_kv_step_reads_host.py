"""What ar_kv_step's kernel reads of the page table before it knows that the
step can be served, run on the host: an entry of the sequence's own row, or
nothing, whatever the lengths are."""

import subprocess

import pytest

from all_reduce_reduction_rank_gb300 import build as arbuild

MOST = 1 << 30


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    exe = tmp_path_factory.mktemp("step") / "step_host"
    src = arbuild.ROOT / "tests" / "step_host.cu"
    subprocess.run([arbuild.nvcc(), *arbuild.ARCH, "-std=c++17", "-I", str(arbuild.INCLUDE), "-I", str(arbuild.CSRC),
                    str(src), "-o", str(exe)], check=True)
    return exe


def cases():
    for shift in (4, 7):
        for stride in (1, 5, 1 << 26, 1 << 27):
            row = min(stride << shift, MOST)
            for old in {0, 1, 15, 16, 17, row - 1, row, row + 1, -1, -16, -2**31, 2**31 - 1, MOST, MOST + 1}:
                for added in (0, 1, 2, 16, row, -1, -2**31, 2**31 - 1):
                    for done in (0, 1):
                        yield old, added, done, stride, shift


def test_entries_read_lie_in_the_row(program):
    todo = list(cases())
    text = "".join("%d %d %d %d %d\n" % c for c in todo)
    out = subprocess.run([str(program)], input=text, capture_output=True, text=True, check=True).stdout.split()
    assert len(out) == 2 * len(todo)
    reads = 0
    for c, entry, bad in zip(todo, map(int, out[::2]), map(int, out[1::2])):
        old, added, done, stride, shift = c
        row, kept = min(stride << shift, MOST), 0 if done else old
        refused = old < 0 or added < 0 or old > row or kept + added > row
        assert bad == refused, c
        if refused or added != 1 or kept % (1 << shift) == 0:
            assert entry == -1, c
        else:
            assert entry == kept >> shift and entry < stride, c
            reads += 1
    assert reads > 20
