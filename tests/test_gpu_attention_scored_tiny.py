"""Scores far below what bounds them and values near the smallest numbers: with
AR_OPT_ATTENTION_PARTS = 2, as in the decode kernel, a row's reference is no larger than its
largest score, whose probability is then 1 or more, and values of 2^-100 keep their bits.

Tolerance, per element: as in test_gpu_attention_scored without the probabilities' rounding, which two parts leave at
u^2 sum p |v|, and 2^-126 a key for products under fp32's normal numbers (the sum that they are divided by is 1 or
more)."""

import numpy as np
import pytest
import torch

import all_reduce_reduction_rank_gb300 as ar
from layer_util import HALF_STEP, Layer, f64
from oracle import layer
from test_gpu_attention_scored import Asked

pytestmark = pytest.mark.gpu

TINY = 2.0**-100
SCALE, CAP, DIM, HEADS = 0.09, 200.0, 128, 4


def fill(L, signs):
    """Keys in the direction of signs[key % 32] times one that every query has, so that scores are near 18 and -18."""
    for r in range(L.n):
        for s, x in enumerate(L.kv):
            sign = torch.tensor([signs[j % 32] for j in range(x)], dtype=torch.float32)[:, None, None]
            L.keys[r][s] = (1.2 * sign + 0.05 * L.keys[r][s].float()).to(torch.bfloat16)
            L.vals[r][s] = (TINY * L.vals[r][s].float()).to(torch.bfloat16)
            for j in range(-(-x // L.page)):
                page, n = int(L.table[s, j]), min(L.page, x - L.page * j)
                for view, src in ((L.kview[r], L.keys[r][s]), (L.vview[r], L.vals[r][s])):
                    view[page, :, :n] = src[L.page * j: L.page * j + n].transpose(0, 1).cuda()


# every score 26 bits below 1, where a cap's bound is as far above it; of 32 keys the one farthest from the row far above
# the others, which a bias of 0.9 a key takes back
FAR = [-1.0] * 32
FIRST = [1.0] + [-1.0] * 31


@pytest.mark.parametrize("what", [{"cap": CAP}, {"cap": CAP, "bias": 0.01}, {"bias": 0.9}, {"cap": CAP, "bias": 0.9}])
@pytest.mark.parametrize("signs", [FAR, FIRST], ids=["far", "first"])
@pytest.mark.parametrize("kernel,max_new", [("decode", 1), ("chunk", 500)])
def test_small_values_keep_their_bits(kernel, max_new, signs, what):
    with Layer(2, 1, DIM, 16, "bf16", [2, 130], [257, 500], max_new=max_new) as L:
        fill(L, signs)
        assert ar.ar_set_option(L.h, ar.AR_OPT_TIMING, 1) == ar.AR_OK
        assert ar.ar_set_option(L.h, ar.AR_OPT_ATTENTION_PARTS, 2) == ar.AR_OK
        cap = what.get("cap", 0.0)
        ask = Asked(L, HEADS, cap=cap, slopes=np.full((2, HEADS), what["bias"]) if "bias" in what else None)
        q, out = [(1.3 + 0.05 * t.float()).to(t.dtype) for t in L.rows(HEADS)], L.rows(HEADS, fill="nan")
        assert ask.call(L, q, out, SCALE) == ar.AR_OK and ar.ar_status(L.h) == ar.AR_OK
        assert ar.ar_timing(L.h)[0][0] == f"attention_{kernel}_scored"
        u, slope = HALF_STEP["bf16"], what.get("bias", 0.0)

        def errors(dots, raw, s, bias):
            of_cap = 1.5 * 2.0**-20 * s + 2.0**-20 * np.log(2) if cap else 0
            return DIM * 2.0**-24 * dots + 2.0**-21 * (raw + 16) + of_cap + 2.0**-22 * (bias + 128 * slope)

        for r in range(2):
            for s, n in enumerate(L.kv):
                a, b = L.starts[s], L.starts[s + 1]
                x = f64(q[r][a:b, : HEADS * DIM]).reshape(b - a, HEADS, DIM)
                want, size, moved = layer.attention_scored(
                    x, f64(L.keys[r][s]), f64(L.vals[r][s]), n - (b - a), SCALE, 0, cap=cap, errors=errors,
                    slopes=None if ask.slopes is None else ask.slopes[r].astype(np.float64))
                tol = u * np.abs(want) + size * (u * u + 2 * (n + 64) * 2.0**-24) + 2 * moved + n * 2.0**-126
                got = f64(out[r][a:b, : HEADS * DIM]).reshape(want.shape)
                assert (np.abs(got - want) <= tol).all(), (r, s, np.max(np.abs(got - want) / tol))
