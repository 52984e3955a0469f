"""ar_paged_attention where its arithmetic can go wrong: NaN in queries and
keys of sequences that are split over CTAs."""

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
