"""Calls whose rows lie in the registered caches are refused before anything is
launched."""

import pytest
import torch

import all_reduce_reduction_rank_gb300 as ar
from layer_util import Layer

pytestmark = pytest.mark.gpu


def test_rows_in_the_caches_are_refused_and_change_nothing():
    with Layer(2, 1, 64, 16, "bf16", [2], [40]) as L:
        q, out = L.rows(4), L.rows(2)
        k, v = [t[:, 128:] for t in q], [t[:, 192:] for t in q]
        before = [c.clone() for c in L.k + L.v]
        cs = torch.zeros((64, 64), device="cuda")
        inside = [c.view(-1)[64:] for c in L.v]

        def append(**x):
            return ar.ar_rope_append(L.handle, L.batch, x.get("q", q), x.get("k", k), x.get("v", v), x.get("out", out), 2,
                                     256, 256, 128, cs, 64, 64, 0)

        for name in ("q", "k", "v", "out"):
            assert append(**{name: inside}) == ar.AR_ERR_INVALID, name
            assert append(**{name: [inside[0], (q if name == "q" else out)[1]]}) == ar.AR_ERR_INVALID, name
        o = L.rows(4)
        call = lambda q, o: ar.ar_paged_attention(L.handle, L.batch, q, o, 4, 256, 256, 0.125, 0)
        assert call(q, inside) == ar.AR_ERR_INVALID
        torch.cuda.synchronize()
        for now, was in zip(L.k + L.v, before):
            assert torch.equal(now.view(torch.int16), was.view(torch.int16))
        assert call(q, o) == ar.AR_OK and append() == ar.AR_OK and ar.ar_status(L.h) == ar.AR_OK
