"""Limits of the layer's calls that only show at their ends, without a GPU."""

import all_reduce_reduction_rank_gb300 as ar
from test_layer_host import append, at, attention, batch, desc, lib  # noqa: F401  (lib: builds and loads the library)


def test_sequences_are_counted_below_2_30():
    # kernels form indices a little past the last sequence in 32 bits
    for seqs in ((1 << 30) + 1, 2**31 - 1):
        assert attention(batch(seqs=seqs)) == ar.AR_ERR_INVALID
        assert append(batch(seqs=seqs)) == ar.AR_ERR_INVALID
    assert attention(batch(seqs=1 << 30)) == ar.AR_OK and append(batch(seqs=1 << 30)) == ar.AR_OK


def test_row_strides_fit_a_tensor_copy():
    # the chunk kernel's copies of the queries take strides below 2^40 bytes
    for stride in (1 << 39, 1 << 40):
        assert attention(batch(tokens=1, seqs=1), qs=stride) == ar.AR_ERR_INVALID
        assert append(batch(tokens=1, seqs=1), qs=stride) == ar.AR_ERR_INVALID
    assert attention(batch(tokens=1, seqs=1), qs=(1 << 39) - 8) == ar.AR_OK


def test_the_scale_is_finite_in_base_2_too():
    # scores are scaled by scale * log2(e), which fp32 must hold
    assert attention(scale=2.3e38) == ar.AR_OK
    for bad in (2.4e38, 3.4e38):
        assert attention(scale=bad) == ar.AR_ERR_INVALID


def test_caches_fit_an_address_space():
    # the kernels form page * page_stride in 64 bits
    ok = lambda d: ar.ar_check_kv(4, d, at(0), at(1))
    assert ok(desc(pages=1 << 20, ps=1 << 38)) == ar.AR_OK
    for bad in ({"pages": 2**31 - 1, "ps": 1 << 38}, {"pages": 1 << 25, "ps": 1 << 38}):
        assert ok(desc(**bad)) == ar.AR_ERR_INVALID, bad
