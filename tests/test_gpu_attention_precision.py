"""The decode kernel feeds the probabilities to the second product as two parts
of the cache's type, the chunk kernel too with AR_OPT_ATTENTION_PARTS = 2, so their
outputs carry no half step of that type for them.

Few keys with nearly equal scores, whose values differ in sign alone: outputs
are small beside sum p |v|, and a half step of the probabilities, u sum p |v|, would
stand out.  Tolerance, per
element: u |out| for the output's rounding; for the probabilities what two parts
leave, u^2 sum p |v| (fp16: or 2^-32 of the largest per key, where numbers end);
scores and sums as in test_gpu_paged_attention."""

import numpy as np
import pytest
import torch

import all_reduce_reduction_rank_gb300 as ar
from layer_util import HALF_STEP, TINY, TORCH, Layer, f64
from oracle import layer
from test_gpu_paged_attention import compare, run


def tolerance(dtype, dim, keys, want, size, dots, top, vmax):
    u = HALF_STEP[dtype]
    d = dim * 2.0**-24 * dots + 2.0**-21 * (top + 16)
    ends = keys * 2.0**-32 * vmax if dtype == "f16" else 0.0
    return u * np.abs(want) + size * (u * u + 2 * d + 2 * (keys + 64) * 2.0**-24) + ends + TINY[dtype]


def alternating(v):
    """One value between 1 and 2 for each column, with the sign of the key's place."""
    sign = torch.tensor([1.0, -1.0]).repeat(v.shape[0] // 2)[:, None, None]
    return ((1 + v[:1].float().abs() % 1) * sign).to(v.dtype)


KEYS = [2, 4, 8]


def check(kernel, group, dim, dtype, max_new, parts):
    with Layer(2, 1, dim, 16, dtype, [1] * len(KEYS), KEYS, seed=group, max_new=max_new) as L:
        for r in range(2):
            for s, n in enumerate(KEYS):
                L.vals[r][s] = alternating(L.vals[r][s])
                for j in range(0, n, 16):
                    L.vview[r][int(L.table[s, j // 16]), :, : min(16, n - j)] = L.vals[r][s][j: j + 16].transpose(0, 1).cuda()
        assert ar.ar_set_option(L.h, ar.AR_OPT_TIMING, 1) == ar.AR_OK
        assert ar.ar_set_option(L.h, ar.AR_OPT_ATTENTION_PARTS, parts) == ar.AR_OK
        q, out = run(L, group, q=[t / 16 for t in L.rows(group)])
        assert ar.ar_timing(L.h)[0][0] == "attention_" + kernel
        for r in range(2):
            for s, n in enumerate(KEYS):
                x = f64(q[r][s: s + 1, : group * dim]).reshape(1, group, dim)
                v = f64(L.vals[r][s])
                want, size, dots, top = layer.attention(x, f64(L.keys[r][s]), v, n - 1, dim**-0.5, 0)
                got = f64(out[r][s: s + 1, : group * dim]).reshape(want.shape)
                tol = tolerance(dtype, dim, n, want, size, dots, top, np.abs(v).max())
                assert (np.abs(got - want) <= tol).all(), (r, s, np.max(np.abs(got - want) / tol))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("group", [1, 4, 8, 12, 16])      # row tiles of 8 and of 16
def test_probabilities_lose_nothing_in_the_decode_kernel(group, dim, dtype):
    check("decode", group, dim, dtype, 1, 1)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("group", [1, 7])
def test_probabilities_lose_nothing_as_two_parts_in_the_chunk_kernel(group, dim, dtype):
    check("chunk", group, dim, dtype, 500, 2)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,dim,window", [("bf16", 128, 0), ("f16", 64, 100), ("f16", 128, 0), ("bf16", 64, 0)])
@pytest.mark.parametrize("new,kv", [([130, 1, 40], [500, 260, 40]), ([513], [640]), ([2, 1], [20000, 3333])])
def test_two_parts_give_the_definition(new, kv, dtype, dim, window):
    first = [max(0, x - q - window + 1) if window else 0 for q, x in zip(new, kv)]
    with Layer(2, 1, dim, 32, dtype, new, kv, max_new=500, first_kept=first) as L:
        assert ar.ar_set_option(L.h, ar.AR_OPT_ATTENTION_PARTS, 2) == ar.AR_OK
        q, out = run(L, 5, window=window)
        compare(L, q, out, 5, dim**-0.5, window)


@pytest.mark.gpu
def test_the_number_of_parts_is_checked():
    with Layer(2, 1, 64, 16, "bf16", [1], [3]) as L:
        for bad in (0, 3, -1):
            assert ar.ar_set_option(L.h, ar.AR_OPT_ATTENTION_PARTS, bad) == ar.AR_ERR_INVALID


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("dim", [64, 128])
def test_probabilities_rounded_once_would_not_pass(dim, dtype):
    # the same check of an fp64 result whose probabilities are rounded once: far outside
    rng = np.random.default_rng(dim)
    dt = TORCH[dtype]
    rounded = lambda a: torch.from_numpy(np.asarray(a)).to(dt).double().numpy()
    for n in KEYS:
        q, k = rounded(rng.standard_normal((1, 8, dim)) / 16), rounded(rng.standard_normal((n, 1, dim)))
        v = alternating(torch.from_numpy(rng.standard_normal((n, 1, dim))).to(dt)).double().numpy()
        want, size, dots, top = layer.attention(q, k, v, n - 1, dim**-0.5, 0)
        s = np.einsum("hd,jd->hj", q[0], k[:, 0]) * dim**-0.5
        p = np.exp(s - s.max(1, keepdims=True))
        once = rounded(np.einsum("hj,jd->hd", rounded(p), v[:, 0]) / p.sum(1, keepdims=True))
        two = rounded(p) + rounded(p - rounded(p))
        twice = rounded(np.einsum("hj,jd->hd", two, v[:, 0]) / p.sum(1, keepdims=True))
        tol = tolerance(dtype, dim, n, want, size, dots, top, np.abs(v).max())[0]
        assert (np.abs(once - want[0]) > 1.5 * tol).any(), n
        assert (np.abs(twice - want[0]) <= tol).all(), n
