"""ar_paged_attention where its arithmetic can go wrong: NaN in queries and
keys of sequences that are split over CTAs, and probabilities far below a row's
largest."""

import numpy as np
import pytest

from layer_util import Layer, f64
from test_gpu_paged_attention import expect, run

pytestmark = pytest.mark.gpu
KERNELS = pytest.mark.parametrize("max_new", [1, 500])   # the decode and the chunk kernel, whatever the batch is


def rows_of(L, out, heads, r, s):
    a, b = L.starts[s], L.starts[s + 1]
    return f64(out[r][a:b, : heads * L.dim]).reshape(b - a, heads, L.dim)


def compare_but(L, q, out, heads, nan_rows):
    """Rows (rank, sequence, token, head) of `nan_rows` are NaN throughout, all others agree with the definition."""
    for r in range(L.n):
        for s in range(len(L.kv)):
            got = rows_of(L, out, heads, r, s)
            with np.errstate(invalid="ignore"):
                want, tol = expect(L, q, heads, L.dim**-0.5, 0, r, s)
            for i in range(got.shape[0]):
                for h in range(heads):
                    if (r, s, i, h) in nan_rows:
                        assert np.isnan(got[i, h]).all(), (r, s, i, h, got[i, h])
                    else:
                        assert (np.abs(got[i, h] - want[i, h]) <= tol[i, h]).all(), (r, s, i, h)


@KERNELS
@pytest.mark.parametrize("dtype,dim", [("bf16", 128), ("f16", 64)])
def test_a_nan_in_a_query_reaches_its_row_and_no_other(dtype, dim, max_new):
    # one sequence over many CTAs, one of a few keys
    heads = 4
    with Layer(2, 1, dim, 128, dtype, [3, 2], [20000, 40], max_new=max_new) as L:
        q = L.rows(heads)
        bad = {(0, 0, 1, 2), (1, 0, 2, 0), (0, 1, 0, 3), (1, 1, 1, 1)}
        for r, s, i, h in bad:
            q[r][L.starts[s] + i, h * dim + 5] = float("nan")
        q, out = run(L, heads, q=q)
        compare_but(L, q, out, heads, bad)


@KERNELS
@pytest.mark.parametrize("first,last", [(0, 128), (0, 640), (0, 1152), (0, 12000), (9000, 20000), (777, 778)])
def test_nan_keys_reach_every_row_that_sees_them(first, last, max_new):
    # with runs of 4 units some cuts fall at 1, 5 and 9 tiles of 128 keys: whole parts see nothing but NaN, others none
    heads, dim, page = 2, 128, 128
    with Layer(2, 1, dim, page, "bf16", [2, 1], [20000, 300], max_new=max_new) as L:
        for r in range(L.n):
            for j in range(first, last):
                if j == first or j % page == 0:
                    p, lo, hi = int(L.table[0, j // page]), j % page, min(page, j % page + last - j)
                    L.kview[r][p, 0, lo:hi] = float("nan")
        q, out = run(L, heads)
        nan_rows = {(r, 0, i, h) for r in range(2) for i in range(2) for h in range(heads)}
        compare_but(L, q, out, heads, nan_rows)


@KERNELS
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("below", [16.0, 25.0, 26.5, 30.0])   # powers of two
def test_weights_far_below_the_largest_still_count(below, dim, max_new):
    """A first key that takes nearly all weight and whose value is 0 (an
    attention sink): the output is what the others' weights, 2^-below each, make
    of their values.  fp16 has no number below 2^-24.  Per key the operand may be
    off by half of that against a largest weight of at least 2^7, so by
    2^-25 2^-7 |v| of the output, beside what `expect` counts."""
    heads, keys = 2, [5000, 60]
    with Layer(2, 1, dim, 64, "f16", [1, 1], keys, max_new=max_new) as L:
        q = L.rows(heads)
        for r in range(L.n):
            q[r][: L.tokens, 0: heads * dim: dim] = 8.0
            for s, n in enumerate(keys):
                k, v = L.keys[r][s], L.vals[r][s].abs() + 0.5
                k *= 2.0**-6
                k[:, :, 0] = 0.0
                k[0] = 0.0
                k[0, :, 0] = below / np.log2(np.e) * dim**0.5 / 8
                v[0] = 0.0
                L.vals[r][s] = v
                for j in range(0, n, L.page):
                    p, m = int(L.table[s, j // L.page]), min(L.page, n - j)
                    L.kview[r][p, :, :m] = k[j: j + m].transpose(0, 1).cuda()
                    L.vview[r][p, :, :m] = v[j: j + m].transpose(0, 1).cuda()
        q, out = run(L, heads, q=q)
        for r in range(L.n):
            for s, n in enumerate(keys):
                want, tol = expect(L, q, heads, dim**-0.5, 0, r, s)
                got = rows_of(L, out, heads, r, s)
                tol = tol + n * 2.0**-32 * f64(L.vals[r][s]).max()
                assert (np.abs(got - want) <= tol).all(), (r, s, got[0, 0, :4], want[0, 0, :4], tol[0, 0, :4])
