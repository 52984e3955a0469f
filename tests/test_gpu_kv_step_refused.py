"""ar_kv_step with lengths that it refuses, at the first, a middle and the last
sequence, each with one new token: the table lies between guard rows, nothing
changes and the status says so."""

import pytest
import torch

import all_reduce_reduction_rank_gb300 as ar
from test_gpu_kv_step import Server, i32

pytestmark = pytest.mark.gpu

PAGE, WIDTH = 16, 5
ROW = PAGE * WIDTH


@pytest.mark.parametrize("seqs", [1, 3, 300, 1024, 2000])
@pytest.mark.parametrize("pad", [0, 3000])       # one CTA, a cluster
@pytest.mark.parametrize("length", [ROW, ROW + 1, -1, -16, -2**31, 2**31 - 1, 1 << 30])
def test_a_refused_length_changes_nothing(length, pad, seqs):
    for at in sorted({0, seqs // 2, seqs - 1}):
        with Server(PAGE, 10, seqs, WIDTH) as x:
            whole = torch.full((seqs + 2, WIDTH), -9, dtype=torch.int32, device="cuda")
            x.table = whole[1:-1]
            x.kv[at] = length
            out = x.outputs(seqs + pad, "apart")
            before = whole.clone(), x.free.clone(), x.kv.clone(), x.count.clone()
            assert x.call(i32([1] * seqs), None, seqs + pad, out) == ar.AR_OK
            assert ar.ar_status(x.h) == ar.AR_ERR_INDEX and ar.ar_status(x.h) == ar.AR_OK
            assert torch.equal(whole, before[0]) and torch.equal(x.free, before[1])
            assert torch.equal(out[1], before[2]) and torch.equal(out[2], before[3])
            assert out[0].tolist() == [0] * (seqs + 1)
            assert out[3].tolist() == [-1] * (seqs + pad) + [-77] * 2 and out[4].tolist() == out[3].tolist()


@pytest.mark.parametrize("length", [ROW - 1, ROW - PAGE + 1])
def test_the_last_tokens_of_a_row(length):
    with Server(PAGE, 30, 3, WIDTH) as x:
        x.step([length] * 3)
        x.step([1] * 3)
