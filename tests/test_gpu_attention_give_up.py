"""ar_paged_attention when a wait for its own copies runs out: every call
ends, reports AR_ERR_WAIT_TIMEOUT, writes nothing but its rows and leaves the
workspace ready for the next one.  The failure is one rank's keys that are
never copied (AR_OPT_ABSENT_RANK); each wait ends after a second."""

import pytest
import torch

import all_reduce_reduction_rank_gb300 as ar
from layer_util import Layer
from test_gpu_paged_attention import compare

pytestmark = pytest.mark.gpu

# keys that fit the ring of tiles; one sequence over many CTAs beside a short one; many; several row tiles each
BATCHES = [([1], [100]), ([3, 2], [20000, 40]), ([1] * 40, list(range(1, 1200, 30))), ([300, 1, 513], [900, 700, 640])]


@pytest.mark.parametrize("max_new", [1, 1000])   # the decode and the chunk kernel, whatever the batch is
@pytest.mark.parametrize("dtype,dim,page,absent", [("bf16", 128, 16, 1), ("f16", 64, 128, 0)])
@pytest.mark.parametrize("new,kv", BATCHES)
def test_a_wait_that_runs_out_ends_the_call_and_nothing_else(new, kv, dtype, dim, page, absent, max_new):
    heads = 4
    with Layer(3, 1, dim, page, dtype, new, kv, max_new=max_new) as L:
        q = L.rows(heads)
        caches = [c.clone() for c in L.k + L.v]
        width = heads * dim

        def call():
            out = L.rows(heads, fill="nan")
            assert ar.ar_paged_attention(L.handle, L.batch, q, out, heads, width, width, dim**-0.5, 0) == ar.AR_OK
            rc, info = ar.ar_status_info(L.h)
            assert info.rank == -1
            for x in out:
                assert torch.isnan(x[L.tokens:].float()).all()
            return out, rc

        first, rc = call()
        assert rc == ar.AR_OK
        assert ar.ar_set_option(L.h, ar.AR_OPT_ABSENT_RANK, absent) == ar.AR_OK
        assert call()[1] == ar.AR_ERR_WAIT_TIMEOUT
        assert ar.ar_set_option(L.h, ar.AR_OPT_ABSENT_RANK, -1) == ar.AR_OK
        for _ in range(2):
            out, rc = call()
            assert rc == ar.AR_OK
            for x, y in zip(out, first):
                assert torch.equal(x[: L.tokens], y[: L.tokens])
        compare(L, q, first, heads, dim**-0.5, 0)
        for now, before in zip(L.k + L.v, caches):
            assert torch.equal(now.view(torch.int16), before.view(torch.int16))
