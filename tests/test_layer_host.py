"""Refusals of the layer's calls, without a GPU: ar_check_block_norm,
ar_check_kv, ar_check_rope_append and ar_check_paged_attention return what the
calls would before they launch anything.  Addresses are made up and never
dereferenced."""

import math

import pytest

import all_reduce_reduction_rank_gb300 as ar
from all_reduce_reduction_rank_gb300 import build as arbuild

BASE, GAP, N = 1 << 40, 1 << 32, 4


@pytest.fixture(scope="module", autouse=True)
def lib():
    arbuild.build()
    return ar.lib()


def at(slot, off=0):
    return [BASE + (slot * N + r) * GAP + off for r in range(N)]


def swap(ptrs, r, p):
    return ptrs[:r] + [p] + ptrs[r + 1:]


def norm(**k):
    T, H = k.get("T", 3), k.get("H", 1024)
    one = BASE + 20 * N * GAP
    return ar.ar_check_block_norm(
        k.get("n", N), k.get("max", 1 << 20), k.get("ins", at(0)), k.get("res", one), k.get("post", one + GAP),
        k.get("gate", one + 2 * GAP), k.get("gs", H), k.get("pre", one + 3 * GAP), k.get("alpha", 1.0),
        k.get("beta", 1.0), k.get("eps", 1e-6), k.get("outs", at(1)), k.get("ro", one + 4 * GAP), T, H,
        k.get("dtype", "bf16"))


def test_block_norm_refusals():
    one = BASE + 20 * N * GAP
    assert norm() == ar.AR_OK
    assert norm(outs=at(0)) == ar.AR_OK and norm(ro=one) == ar.AR_OK          # in place
    assert norm(post=None) == ar.AR_OK and norm(gate=None, gs=0) == ar.AR_OK
    assert norm(gs=0) == ar.AR_OK and norm(T=0) == ar.AR_OK
    for bad in ({"n": 1}, {"n": 17}, {"dtype": 3}, {"H": 0}, {"H": 1004}, {"H": 65544}, {"eps": -1.0},
                {"eps": math.nan}, {"eps": math.inf}, {"alpha": math.nan}, {"beta": math.inf}, {"res": None},
                {"pre": None}, {"ro": None}, {"gs": 1020}, {"gs": 512}, {"ins": swap(at(0), 2, None)},
                {"outs": swap(at(1), 1, at(1)[0])}, {"ro": at(1)[3]}, {"ro": at(0)[3]}, {"pre": at(1)[0] + 64},
                {"post": at(1)[2] + 64}, {"gate": one + 4 * GAP + 16}, {"res": at(1)[0]}):
        assert norm(**bad) == ar.AR_ERR_INVALID, bad
    for bad in ({"res": one + 8}, {"post": one + GAP + 4}, {"gate": one + 2 * GAP + 2}, {"pre": one + 3 * GAP + 8},
                {"ro": one + 8 + GAP * 4}, {"ins": at(0, 2)}):
        assert norm(**bad) == ar.AR_ERR_ALIGN, bad
    assert norm(T=600) == ar.AR_ERR_TOO_LARGE


def desc(**k):
    D, P, H = k.get("dim", 128), k.get("page", 16), k.get("heads", 2)
    return ar.KvDesc(ar._dtype(k.get("dtype", "bf16")), H, D, P, k.get("pages", 100), k.get("ps", H * P * D),
                     k.get("hs", P * D), k.get("ts", D))


def test_cache_refusals():
    ok = lambda d, ks=None, vs=None, n=N: ar.ar_check_kv(n, d, ks or at(0), vs or at(1))
    assert ok(desc()) == ar.AR_OK
    assert ok(desc(ps=16 * 2 * 128 * 2, hs=128, ts=256)) == ar.AR_OK   # [page][2][slot][head][d]
    for bad in ({"dtype": "f32"}, {"dim": 96}, {"dim": 256}, {"page": 8}, {"page": 48}, {"page": 256}, {"heads": 0},
                {"heads": 1025}, {"pages": 0}, {"pages": 1 << 31}, {"ps": 0}, {"hs": 12}, {"ts": 64}, {"ts": 130},
                {"ps": 1 << 39}):
        assert ok(desc(**bad)) == ar.AR_ERR_INVALID, bad
    assert ok(desc(), n=1) == ar.AR_ERR_INVALID
    assert ok(desc(), swap(at(0), 1, None)) == ar.AR_ERR_INVALID
    assert ok(desc(), swap(at(0), 1, at(0)[0])) == ar.AR_ERR_INVALID
    assert ok(desc(), at(0), swap(at(1), 2, at(0)[2])) == ar.AR_ERR_INVALID
    assert ok(desc(), at(0, 8)) == ar.AR_ERR_ALIGN


def batch(**k):
    one = BASE + 30 * N * GAP
    return ar.ar_batch(k.get("tokens", 5), k.get("seqs", 2), k.get("most", 4), k.get("q_start", one),
                       k.get("kv_len", one + GAP), k.get("table", one + 2 * GAP), k.get("stride", 7))


BAD_BATCHES = ({"seqs": 0}, {"seqs": -1}, {"most": 0}, {"q_start": None}, {"kv_len": None}, {"table": None},
               {"stride": 0}, {"stride": (1 << 27) + 1}, {"tokens": (1 << 30) + 1})


def attention(b=None, **k):
    row = 8 * 128
    return ar.ar_check_paged_attention(k.get("n", N), k.get("desc", desc()), b or batch(), k.get("q", at(2)),
                                       k.get("out", at(3)), k.get("heads", 8), k.get("qs", row), k.get("os", row),
                                       k.get("scale", 0.1), k.get("window", 0))


def test_attention_refusals():
    assert attention() == ar.AR_OK and attention(window=7) == ar.AR_OK and attention(batch(tokens=0)) == ar.AR_OK
    assert attention(qs=2048, out=at(2, 2048), os=2048) == ar.AR_OK      # columns of one allocation
    for bad in BAD_BATCHES:
        assert attention(batch(**bad)) == ar.AR_ERR_INVALID, bad
    assert attention(batch(q_start=BASE + 2)) == ar.AR_ERR_ALIGN
    for bad in ({"n": 17}, {"heads": 7}, {"heads": 0}, {"heads": 130}, {"qs": 1016}, {"os": 1028}, {"scale": 0.0},
                {"scale": -1.0}, {"scale": math.nan}, {"scale": math.inf}, {"window": -1}, {"out": at(2)},
                {"out": at(2, 512)}, {"q": swap(at(2), 0, None)}, {"out": swap(at(3), 1, at(3)[0])},
                {"desc": desc(dim=96)}, {"qs": 1 << 41}):
        assert attention(**bad) == ar.AR_ERR_INVALID, bad
    assert attention(q=at(2, 8)) == ar.AR_ERR_ALIGN and attention(out=at(3, 4)) == ar.AR_ERR_ALIGN


def append(b=None, **k):
    row = 12 * 128
    return ar.ar_check_rope_append(k.get("n", N), desc(), b or batch(), k.get("q", at(2)), k.get("k", at(2, 2048)),
                                   k.get("v", at(2, 2560)), k.get("out", at(3)), k.get("heads", 8), k.get("qs", row),
                                   k.get("ks", row), k.get("os", 1024), k.get("cs", BASE + 40 * N * GAP),
                                   k.get("mp", 100), k.get("rot", 128), k.get("il", 0))


def test_append_refusals():
    assert append() == ar.AR_OK and append(il=1) == ar.AR_OK and append(rot=0, cs=None, mp=0) == ar.AR_OK
    assert append(q=None, out=None) == ar.AR_OK and append(batch(tokens=0)) == ar.AR_OK
    assert append(out=at(2), os=12 * 128) == ar.AR_OK                     # in place
    for bad in BAD_BATCHES:
        assert append(batch(**bad)) == ar.AR_ERR_INVALID, bad
    for bad in ({"n": 0}, {"rot": 8}, {"rot": 144}, {"rot": -16}, {"il": 2}, {"cs": None}, {"mp": 0}, {"out": None},
                {"q": None}, {"heads": 0}, {"qs": 1000}, {"ks": 200}, {"os": 1020}, {"k": swap(at(4), 3, None)},
                {"out": at(2)}, {"out": at(2, 2048), "os": 12 * 128}, {"out": swap(at(3), 0, at(3)[2])}):
        assert append(**bad) == ar.AR_ERR_INVALID, bad
    for bad in ({"q": at(2, 2)}, {"k": at(4, 8)}, {"v": at(4, 8)}, {"out": at(3, 8)}, {"cs": BASE + 4}):
        assert append(**bad) == ar.AR_ERR_ALIGN, bad
