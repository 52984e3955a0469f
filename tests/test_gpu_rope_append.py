"""ar_rope_append against the 64-bit definition.  Values are copied bit for
bit; a rotated element is off by half a step of its type and by the fp32
products' 4 roundings, 4 2^-24 (|x1 c| + |x2 s|)."""

import numpy as np
import pytest
import torch

import all_reduce_reduction_rank_gb300 as ar
from layer_util import HALF_STEP, TINY, TORCH, Layer, f64
from oracle import layer

pytestmark = pytest.mark.gpu


def table(positions, R):
    ang = np.arange(positions)[:, None] * 10000.0 ** (-np.arange(0, R, 2) / max(R, 1))
    return torch.from_numpy(np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)).cuda()


def near(got, want, size, dtype):
    tol = HALF_STEP[dtype] * np.abs(want) + 4 * 2.0**-24 * size + TINY[dtype]
    return (np.abs(got - want) <= tol).all()


def check(n, q_heads, kv_heads, dim, page, dtype, new, kv, R, interleaved, *, order="head", pad=0, mode="out", stream=None):
    # the caches start with NaN everywhere that this call does not write
    with Layer(n, kv_heads, dim, page, dtype, new, kv, order=order,
               first_kept=[10**9] * len(kv)) as L:
        at = 0
        for s, x in enumerate(kv):   # every page of the tokens' range
            for j in range(-(-x // page)):
                L.table[s, j] = at
                at += 1
        heads = (q_heads + 2 * kv_heads)
        stride = heads * dim + pad
        x = L.rows(heads, stride)
        k, v = [t[:, q_heads * dim:] for t in x], [t[:, (q_heads + kv_heads) * dim:] for t in x]
        src = [t.clone() for t in x]
        out, os = (x, stride) if mode == "in place" else (L.rows(q_heads, fill="nan"), q_heads * dim)
        cs = table(max(kv) + 1, R) if R else None
        rc = ar.ar_rope_append(L.handle, L.batch, None if mode == "no q" else x, k, v, None if mode == "no q" else out,
                               q_heads, stride, stride, os, cs, max(kv) + 1 if R else 0, R, interleaved, stream)
        assert rc == ar.AR_OK and ar.ar_status(L.h) == ar.AR_OK
        want_k = [torch.full_like(t, float("nan")) for t in L.kview]
        want_v = [torch.full_like(t, float("nan")) for t in L.vview]
        for r in range(n):
            for t, (s, pos) in enumerate(layer.positions(L.starts, kv)):
                row = f64(src[r][t, : heads * dim]).reshape(heads, dim)
                p, slot = int(L.table[s, pos // page]), pos % page
                turn = (lambda a: layer.rotate(a, cs[pos].cpu().numpy(), interleaved)) if R else \
                    (lambda a: (a, 0 * a))
                if mode != "no q":
                    want, size = turn(row[:q_heads])
                    assert near(f64(out[r][t, : q_heads * dim]).reshape(want.shape), want, size, dtype)
                want, size = turn(row[q_heads: q_heads + kv_heads])
                got = L.kview[r][p, :, slot]
                assert near(f64(got), want, size, dtype)
                if R < dim:
                    assert torch.equal(got[:, R:], src[r][t, q_heads * dim: (q_heads + kv_heads) * dim].view(-1, dim)[:, R:])
                want_k[r][p, :, slot] = got
                want_v[r][p, :, slot] = src[r][t, (q_heads + kv_heads) * dim: heads * dim].view(-1, dim)
            # values bit for bit, every other slot untouched
            for got, want in ((L.kview[r], want_k[r]), (L.vview[r], want_v[r])):
                assert torch.equal(got.contiguous().view(torch.int16), want.contiguous().view(torch.int16))
            if mode == "out":
                assert torch.isnan(out[r][L.tokens:].float()).all()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("interleaved", [0, 1])
@pytest.mark.parametrize("dim,R", [(64, 64), (128, 128), (128, 64), (64, 16), (128, 48), (64, 0)])
def test_rotations(dim, R, interleaved, dtype):
    check(2, 3, 2, dim, 16, dtype, [1, 5, 0, 18], [7, 33, 4, 18], R, interleaved)


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("order", ["head", "slot", "pair"])
def test_pages_and_orders(page, order):
    check(3, 4, 1, 128, page, "bf16", [1, 70, 1], [1, 200, 129], 128, 0, order=order, pad=8)


@pytest.mark.parametrize("mode", ["in place", "no q"])
def test_in_place_and_without_queries(mode):
    check(2, 5, 2, 64, 16, "f16", [3, 20], [3, 40], 64, 1, mode=mode)


def test_many_sequences_and_heads():
    rng = np.random.default_rng(3)
    new = [int(x) for x in rng.integers(0, 3, 90)]
    kv = [int(q + x) for q, x in zip(new, rng.integers(0, 40, 90))]
    check(2, 40, 3, 64, 32, "bf16", new, kv, 64, 0)


@pytest.mark.parametrize("q_heads,kv_heads,dim,R,interleaved", [(7, 1, 64, 32, 1), (4, 2, 128, 128, 0), (40, 3, 128, 64, 0),
                                                               (1, 1, 64, 64, 1), (70, 2, 64, 48, 0)])
def test_many_tokens(q_heads, kv_heads, dim, R, interleaved):
    # over 1024 tokens x ranks: 4 heads a thread, up to 4 tokens a CTA, or several CTAs a token
    check(2, q_heads, kv_heads, dim, 64, "bf16", [301, 1, 0, 250], [301, 77, 5, 400], R, interleaved, pad=8)


def test_another_stream():
    s = torch.cuda.Stream()
    check(2, 2, 1, 64, 16, "bf16", [2], [9], 64, 0, stream=s)


def test_bad_entries_reach_no_memory_and_are_reported():
    def case(spoil, left, max_positions=64):
        """`left`: packed tokens that are left out."""
        with Layer(2, 1, 64, 16, "bf16", [1, 2], [20, 40]) as L:
            before = [[t.clone() for t in c] for c in (L.k, L.v)]
            spoil(L)
            x = L.rows(4)
            out = L.rows(2, fill="nan")
            k, v = [t[:, 128:] for t in x], [t[:, 192:] for t in x]
            assert ar.ar_rope_append(L.handle, L.batch, x, k, v, out, 2, 256, 256, 128, table(64, 64), max_positions,
                                     64, 0) == ar.AR_OK
            assert ar.ar_status(L.h) == ar.AR_ERR_INDEX
            assert ar.ar_status(L.h) == ar.AR_OK
            for r in range(2):
                wrote = [t for t in range(3) if not torch.isnan(out[r][t].float()).any()]
                assert wrote == [t for t in range(3) if t not in left]
                assert torch.isnan(out[r][3:].float()).all()
                changed = sum(int((a.view(torch.int16) != b.view(torch.int16)).any(-1).sum())
                              for a, b in ((L.v[r], before[1][r]),))
                assert changed == len(wrote)

    case(lambda L: L.table[0].fill_(L.pages), [0])
    case(lambda L: L.table[1].fill_(-1), [1, 2])
    case(lambda L: L.kv_len[1:].fill_(1), [1])            # the first of its tokens has position -1
    case(lambda L: L.kv_len[1:].fill_(1 << 30), [1, 2])
    case(lambda L: L.q_start[2:].fill_(9), [1, 2])
    case(lambda L: None, [2], max_positions=39)
