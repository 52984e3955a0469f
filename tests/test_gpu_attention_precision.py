"""The decode kernel feeds the probabilities to the second product as two parts
of the cache's type, so its outputs carry no half step of that type for them.

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
from test_gpu_paged_attention import run


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


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("group", [1, 4, 8, 12, 16])      # row tiles of 8 and of 16
def test_probabilities_lose_nothing_in_the_decode_kernel(group, dim, dtype):
    with Layer(2, 1, dim, 16, dtype, [1] * len(KEYS), KEYS, seed=group) as L:
        for r in range(2):
            for s, n in enumerate(KEYS):
                L.vals[r][s] = alternating(L.vals[r][s])
                for j in range(0, n, 16):
                    L.vview[r][int(L.table[s, j // 16]), :, : min(16, n - j)] = L.vals[r][s][j: j + 16].transpose(0, 1).cuda()
        assert ar.ar_set_option(L.h, ar.AR_OPT_TIMING, 1) == ar.AR_OK
        q, out = run(L, group, q=[t / 16 for t in L.rows(group)])
        assert ar.ar_timing(L.h)[0][0] == "attention_decode"
        for r in range(2):
            for s, n in enumerate(KEYS):
                x = f64(q[r][s: s + 1, : group * dim]).reshape(1, group, dim)
                v = f64(L.vals[r][s])
                want, size, dots, top = layer.attention(x, f64(L.keys[r][s]), v, n - 1, dim**-0.5, 0)
                got = f64(out[r][s: s + 1, : group * dim]).reshape(want.shape)
                tol = tolerance(dtype, dim, n, want, size, dots, top, np.abs(v).max())
                assert (np.abs(got - want) <= tol).all(), (r, s, np.max(np.abs(got - want) / tol))


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
