"""ar_paged_attention_scored: what no row sees leaves the results' bits alone,
slots behind a sequence's keys and before its first document, stale tiles of
calls before, and the queries of rows that are padding."""

import pytest
import torch

import all_reduce_reduction_rank_gb300 as ar
from layer_util import Layer
from test_gpu_attention_scored import Asked, slopes_of

pytestmark = pytest.mark.gpu

ASKED = {"masks": {}, "cap": {"cap": 30.0}, "bias": {"bias": True}, "both": {"cap": 30.0, "bias": True}}
FILLS = (0.0, 300.0, -40.0, float("inf"), float("nan"))
PAD = 150


def asked(L, heads, what):
    kw = dict(ASKED[what])
    slopes = slopes_of(L.n, heads) / 8 if kw.pop("bias", False) else None
    return Asked(L, heads, slopes=slopes, first=[min(130, k - q) for q, k in zip(L.new, L.kv) for _ in range(q)] + [0] * PAD,
                 prefix=[0] * len(L.kv), **kw)


def run(L, ask, q):
    out = L.rows(ask.heads, fill="nan")
    assert ask.call(L, q, out, L.dim**-0.5) == ar.AR_OK and ar.ar_status(L.h) == ar.AR_OK
    n = sum(L.new)
    return [t[:n].clone().view(torch.int16) for t in out]


@pytest.mark.parametrize("what", list(ASKED))
@pytest.mark.parametrize("dtype,dim", [("bf16", 128), ("f16", 64), ("f16", 128)])
@pytest.mark.parametrize("max_new", [1, 500])
def test_hidden_slots_and_padding_do_not_matter(max_new, dtype, dim, what):
    new, kv = [70, 1, 200, 33], [300, 137, 333, 1000]
    with Layer(2, 1, dim, 32, dtype, new, kv, max_new=max_new) as L:
        L.tokens = L.batch.tokens = sum(new) + PAD
        ask, q = asked(L, 5, what), L.rows(5)
        unused = [torch.isnan(t) for t in L.k]           # slots of the pages that no key is in
        want = None
        for fill in FILLS:
            for t, at in zip(L.k + L.v, unused + unused):
                t.masked_fill_(at, fill)
            for t in q:
                t[sum(new): L.tokens] = fill
            got = run(L, ask, q)
            want = got if want is None else want
            assert all(torch.equal(x, y) for x, y in zip(got, want)), fill


@pytest.mark.parametrize("what", list(ASKED))
@pytest.mark.parametrize("max_new", [1, 500])
def test_tiles_of_earlier_calls_do_not_matter(max_new, what):
    # pages of 16: most of the last tile of each sequence is not copied, what another call left there remains
    new, kv = [70, 1, 200, 33], [300, 133, 262, 1030]
    with Layer(2, 1, 128, 16, "bf16", new, kv, max_new=max_new) as L, \
            Layer(2, 1, 128, 16, "bf16", [300, 300], [2000, 3000], max_new=max_new) as M:
        ask, q = asked(L, 5, what), L.rows(5)
        other, p = asked(M, 5, what), M.rows(5)
        want = None
        for fill in FILLS[:3]:
            for t in M.k:
                t.fill_(fill)
            run(M, other, p)
            got = run(L, ask, q)
            want = got if want is None else want
            assert all(torch.equal(x, y) for x, y in zip(got, want)), fill
