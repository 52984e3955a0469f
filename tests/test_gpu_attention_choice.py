"""Which kernel ar_paged_attention takes: the decode kernel while one pass over
the keys (two for heads of 64) serves all rows of a sequence, a row tile being
whole tokens of up to 16 heads."""

import pytest

import all_reduce_reduction_rank_gb300 as ar
from layer_util import Layer
from test_gpu_paged_attention import compare, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dim,group,new,kernel", [
    (128, 8, 1, "decode"), (128, 16, 1, "decode"), (128, 5, 3, "decode"), (128, 6, 3, "chunk"), (128, 17, 1, "chunk"),
    (128, 8, 3, "chunk"), (64, 8, 4, "decode"), (64, 32, 1, "decode"), (64, 6, 4, "decode"),
    (64, 9, 3, "chunk"), (64, 6, 5, "chunk"), (64, 33, 1, "chunk"), (64, 8, 5, "chunk")])
def test_the_kernel_follows_the_passes_over_the_keys(dim, group, new, kernel):
    with Layer(2, 1, dim, 16, "bf16", [new, 1], [200, 70]) as L:
        assert ar.ar_set_option(L.h, ar.AR_OPT_TIMING, 4) == ar.AR_OK
        q, out = run(L, group)
        assert [r[0] for r in ar.ar_timing(L.h)] == ["attention_" + kernel]
        compare(L, q, out, group, dim**-0.5, 0)
