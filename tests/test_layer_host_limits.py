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


def apart(rows, d=None, ks=None, vs=None, row=1024, stride=1024, tokens=5):
    return ar.ar_check_rows_apart(4, d or desc(), ks or at(0), vs or at(1), rows, row, stride, tokens)


def test_rows_in_a_cache_are_refused():
    page = 2 * 16 * 128 * 2                       # bytes of a page of desc(), 100 of them
    assert apart(at(2)) == ar.AR_OK and apart(at(0, 100 * page)) == ar.AR_OK and apart(at(0), tokens=0) == ar.AR_OK
    for off in (0, 16, 50 * page, 100 * page - 16):
        assert apart(at(0, off)) == ar.AR_ERR_INVALID and apart(at(1, off)) == ar.AR_ERR_INVALID
    for off in (-5 * 2048 + 16, -16):             # rows that begin before a cache and end in it
        assert apart(at(0, off)) == ar.AR_ERR_INVALID
    assert apart(at(0, -5 * 2048)) == ar.AR_OK
    for r in range(4):                            # one rank's rows in another rank's cache
        rows = at(2)
        rows[r] = at(1)[(r + 1) % 4] + 4 * page
        assert apart(rows) == ar.AR_ERR_INVALID
    assert apart(at(0, 8)) == ar.AR_ERR_ALIGN and apart(at(2), stride=1000) == ar.AR_ERR_INVALID


def test_rows_between_the_pages_of_a_cache_are_apart():
    # one allocation of pages with room behind each: [page][2 x 16 x 128 of K, as much of V, 2048 elements more]
    d = desc(ps=2 * 4096 + 2048)
    step = 2 * (2 * 4096 + 2048)
    vs, rows = at(0, 2 * 4096), at(0, 4 * 4096)
    assert ar.ar_check_kv(4, d, at(0), vs) == ar.AR_OK
    for tokens in (1, 5, 100, 130):               # more and fewer rows than pages, one row behind a page
        assert apart(rows, d, vs=vs, stride=step // 2, tokens=tokens) == ar.AR_OK
        assert apart([p + 2048 + 16 for p in rows], d, vs=vs, stride=step // 2, tokens=tokens) == (
            ar.AR_ERR_INVALID if tokens > 0 else ar.AR_OK)
    # rows that follow one another reach the next page
    assert apart(rows, d, vs=vs, tokens=2) == ar.AR_OK and apart(rows, d, vs=vs, tokens=3) == ar.AR_ERR_INVALID


def test_caches_that_share_elements_are_refused():
    page, kb = 2 * 16 * 128, 2                       # elements of a page of K, bytes of one
    ok = lambda d, ks, vs: ar.ar_check_kv(4, d, ks, vs)
    near = lambda off: [p + off * kb for p in at(0)]
    # values behind the keys, right behind and one vector too near; keys in the values' last page
    assert ok(desc(), at(0), near(100 * page)) == ar.AR_OK
    for off in (100 * page - 8, 99 * page + 64, 8, -8, 128, -100 * page + 8):
        assert ok(desc(), at(0), near(off)) == ar.AR_ERR_INVALID, off
    assert ok(desc(), at(0), near(-100 * page)) == ar.AR_OK
    # two ranks' keys
    ks = at(0)
    ks[3] = ks[1] + 5 * page * kb
    assert ok(desc(), ks, at(1)) == ar.AR_ERR_INVALID
    # keys and values side by side in each page, in each slot, in each head
    side = {"page": (dict(ps=2 * page), page), "slot": (dict(ps=2 * page, ts=512, hs=128), 256),
            "head": (dict(ps=2 * page, ts=128, hs=2 * 16 * 128), 16 * 128),
            "head of a slot": (dict(ps=2 * page, ts=512, hs=256), 128)}
    for name, (strides, off) in side.items():
        assert ok(desc(**strides), at(0), near(off)) == ar.AR_OK, name
        for more in (8, -8, 120):
            assert ok(desc(**strides), at(0), near(off + more)) == ar.AR_ERR_INVALID, (name, more)


def test_caches_whose_own_slots_overlap_are_refused():
    ok = lambda **k: ar.ar_check_kv(4, desc(**k), at(0), at(1))
    assert ok(heads=1, hs=8) == ar.AR_OK and ok(pages=1, ps=8) == ar.AR_OK     # no second head, no second page
    assert ok(ts=256, hs=128, ps=16 * 256) == ar.AR_OK
    for bad in (dict(hs=8), dict(hs=120), dict(ps=2 * 16 * 128 - 8), dict(ps=120), dict(ts=136), dict(ts=256, hs=136)):
        assert ok(**bad) == ar.AR_ERR_INVALID, bad
