"""ar_allreduce_block_norm against the 64-bit definition.  With u half a step
of the type and e = 2^-24 of fp32: a value of r is off by u |r| and, before
that rounding, by (n + 24) e per unit of its terms (the rank sum, six
products, and a mean of squares summed over threads, warps and CTAs, whose
relative error is under 32 e and halves under the root); y adds the
same again, scaled like r."""

import numpy as np
import pytest
import torch

import all_reduce_reduction_rank_gb300 as ar
from gpu_util import Handle
from layer_util import HALF_STEP, TINY, TORCH, f64
from oracle import layer

pytestmark = pytest.mark.gpu
E = {"f32": 4, "bf16": 2, "f16": 2}


class Case:
    def __init__(self, n, T, H, dtype, gate, post, seed=0):
        g = torch.Generator().manual_seed(seed)
        dt = TORCH[dtype]
        make = lambda *s: torch.randn(s, generator=g).to(dt).cuda()
        nan = lambda *s: torch.full(s, float("nan"), dtype=dt, device="cuda")
        self.n, self.T, self.H, self.dtype = n, T, H, dtype
        self.ins = [make(T, H) for _ in range(n)]
        self.res, self.pre = make(T, H), make(H)
        self.post = make(H) if post else None
        self.stride = {"token": H, "wide": 3 * H, "shared": 0, None: 0}[gate]
        self.wide = make(T, 3 * H) if gate == "wide" else make(T if gate == "token" else 1, H)
        self.gate = self.wide if gate else None       # "wide": a column block of a wider buffer
        # one spare row after each output
        self.outs, self.ro = [nan(T + 1, H) for _ in range(n)], nan(T + 1, H)

    def call(self, h, stream=None, alpha=0.75, beta=1.5, eps=1e-5):
        return ar.ar_allreduce_block_norm(h, self.ins, self.res, self.post, self.gate, self.stride, self.pre, alpha,
                                          beta, eps, self.outs, self.ro, self.T, self.H, self.dtype, stream)

    def want(self, alpha=0.75, beta=1.5, eps=1e-5):
        f = lambda t: None if t is None else f64(t)
        gate = f(self.gate)
        if gate is not None:
            gate = gate[:, : self.H]
        xs = [f(x[: self.T]) for x in self.ins]      # another case's outputs have a spare row
        y, r, size = layer.block_norm(xs, f(self.res[: self.T]), f(self.post), gate, f(self.pre), alpha, beta, eps)
        u, e = HALF_STEP[self.dtype], 2.0**-24
        raw = (self.n + 24) * e * size
        scale = np.abs(f(self.pre)) / np.sqrt((r * r).mean(-1, keepdims=True) + eps)
        tiny = TINY[self.dtype]
        return y, r, u * np.abs(y) + scale * raw + 24 * e * np.abs(y) + tiny, u * np.abs(r) + raw + tiny

    def check(self, **k):
        y, r, ty, tr = self.want(**k)
        got = f64(self.ro[: self.T])
        assert (np.abs(got - r) <= tr).all(), np.max(np.abs(got - r) / tr)
        for o in self.outs:
            got = f64(o[: self.T])
            assert (np.abs(got - y) <= ty).all(), np.max(np.abs(got - y) / ty)
            assert torch.equal(o[: self.T], self.outs[0][: self.T])
        for o in self.outs + [self.ro]:
            assert torch.isnan(o[self.T:].float()).all()


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("gate,post", [("token", True), ("shared", True), (None, True), ("wide", False), (None, False)])
@pytest.mark.parametrize("n,T,H", [(8, 1, 4096), (2, 5, 8), (3, 7, 520), (16, 3, 8200), (4, 33, 2048)])
def test_block_norm(n, T, H, gate, post, dtype):
    c = Case(n, T, H, dtype, gate, post, seed=T + H)
    with Handle(n, T * H * E[dtype]) as h:
        assert c.call(h) == ar.AR_OK and ar.ar_status(h) == ar.AR_OK
        t = ar.ar_traffic(h)
        S, W = T * H * E[dtype], H * E[dtype]
        extra = W * (1 + post) + {"token": S, "wide": S, "shared": W, None: 0}[gate]
        assert (t.op, t.hbm_read_bytes, t.hbm_write_bytes) == (ar.AR_OP_ALLREDUCE_BLOCK_NORM, (n + 1) * S + extra,
                                                               (n + 1) * S)
    c.check()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("H", [16384, 40000, 65536])
def test_long_rows(H, dtype):
    c = Case(4, 3, H, dtype, "shared", True)
    with Handle(4, 3 * H * E[dtype]) as h:
        assert c.call(h) == ar.AR_OK and ar.ar_status(h) == ar.AR_OK
    c.check()


@pytest.mark.parametrize("n,T,H", [(8, 300, 1024), (2, 1000, 4096), (8, 700, 8192), (5, 333, 200)])
def test_many_tokens(n, T, H):
    c = Case(n, T, H, "bf16", "token", True)
    with Handle(n, T * H * 2) as h:
        assert c.call(h) == ar.AR_OK and ar.ar_status(h) == ar.AR_OK
    c.check()


def test_in_place_and_other_factors():
    c = Case(4, 6, 1024, "bf16", "token", True)
    want = c.want(alpha=-1.0, beta=0.25, eps=0.0)
    pad = lambda t: torch.cat([t, torch.full_like(t[:1], float("nan"))])
    c.outs, c.ro = [pad(x) for x in c.ins], pad(c.res)
    c.ins, c.res = c.outs, c.ro
    with Handle(4, 6 * 1024 * 2) as h:
        assert c.call(h, alpha=-1.0, beta=0.25, eps=0.0) == ar.AR_OK and ar.ar_status(h) == ar.AR_OK
    c.want = lambda **k: want
    c.check()


def test_rows_of_zeros_and_no_tokens():
    c = Case(2, 2, 64, "f16", "shared", True)
    for t in c.ins + [c.res]:
        t.zero_()
    with Handle(2, 1 << 12) as h:
        assert c.call(h) == ar.AR_OK and ar.ar_status(h) == ar.AR_OK
        c.check()
        c.T = 0
        for o in c.outs + [c.ro]:
            o.fill_(float("nan"))
        assert c.call(h) == ar.AR_OK and ar.ar_traffic(h).launches == 0
        torch.cuda.synchronize()
        c.T = 0
        assert all(torch.isnan(o.float()).all() for o in c.outs)
        c.T = 100
        assert c.call(h) == ar.AR_ERR_TOO_LARGE


@pytest.mark.parametrize("pdl", [0, 1])
@pytest.mark.parametrize("T,H", [(1, 4096), (24, 8192)])
def test_chained_calls_in_a_graph_read_their_predecessors(T, H, pdl):
    # call k + 1 takes call k's outputs and residual; the graph's outputs equal the eager chain's
    n, K = 4, 4
    cases = [Case(n, T, H, "bf16", "shared", True, seed=7) for _ in range(K)]
    for a, b in zip(cases, cases[1:]):
        b.ins, b.res = a.outs, a.ro
    with Handle(n, T * H * 2, pdl=pdl) as h:
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        for c in cases:
            assert c.call(h, s) == ar.AR_OK
        s.synchronize()
        eager = [[o.clone() for o in c.outs + [c.ro]] for c in cases]
        for c in cases:
            c.check()
        for c in cases:
            for o in c.outs + [c.ro]:
                o.fill_(float("nan"))
        g = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g, stream=s):
            for c in cases:
                assert c.call(h, s) == ar.AR_OK
        g.replay()
        torch.cuda.synchronize()
        assert ar.ar_status(h) == ar.AR_OK
    for c, e in zip(cases, eager):
        for o, w in zip(c.outs + [c.ro], e):
            assert torch.equal(o[:T], w[:T])
