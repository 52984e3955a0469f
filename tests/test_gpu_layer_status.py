"""What ar_status_info says of the layer's calls."""

import pytest

import all_reduce_reduction_rank_gb300 as ar
from layer_util import Layer

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("max_new", [1, 500])
def test_an_entry_out_of_range_names_no_rank(max_new):
    with Layer(2, 1, 64, 16, "bf16", [1, 1], [50, 70], max_new=max_new) as L:
        L.table[1].fill_(L.pages)
        q, out = L.rows(4), L.rows(4, fill="nan")
        assert ar.ar_paged_attention(L.handle, L.batch, q, out, 4, 256, 256, 0.125, 0) == ar.AR_OK
        rc, info = ar.ar_status_info(L.h)
        assert rc == info.code == ar.AR_ERR_INDEX
        assert (info.rank, info.line, info.lines_skipped) == (-1, 0, 0)
        rc, info = ar.ar_status_info(L.h)
        assert rc == ar.AR_OK and info.rank == -1
