"""One tensor-parallel attention block on n emulated ranks, decode steps and
prefill chunks alike, with every call of the library where a layer uses it:

    qkv = y W_qkv                    (per rank: its share of the heads)
    ar_rope_append                   rotate q and k, append k and v to the paged caches
    ar_paged_attention               the new tokens over the caches
    part = out W_o                   (per rank: a partial sum of the block's output)
    ar_allreduce_block_norm          sum of the parts, norm, gate, residual, next norm

    python examples/tp_layer.py [--ranks 8] [--steps 4] [--check]

--check compares every step with the same block in fp64 and exits 1 beyond
bf16's accuracy.
"""

import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import all_reduce_reduction_rank_gb300 as ar  # noqa: E402

PAGE, DIM, EPS, BETA = 32, 128, 1e-6, 0.5


class Layer:
    """The block's weights, per rank, and its caches."""

    def __init__(self, n, hidden, heads, kv_heads, pages, max_tokens, max_positions, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        make = lambda *s, scale=1.0: (torch.randn(s, generator=g, device="cuda") * scale).bfloat16()
        self.n, self.hidden, self.q, self.kv = n, hidden, heads // n, kv_heads // n
        row = (self.q + 2 * self.kv) * DIM
        self.w_qkv = [make(hidden, row, scale=hidden**-0.5) for _ in range(n)]
        self.w_o = [make(self.q * DIM, hidden, scale=(heads * DIM) ** -0.5) for _ in range(n)]
        self.post, self.pre, self.gate = 1 + make(hidden, scale=0.1), 1 + make(hidden, scale=0.1), make(hidden)
        cache = lambda: [torch.zeros((pages, self.kv, PAGE, DIM), dtype=torch.bfloat16, device="cuda") for _ in range(n)]
        self.k, self.v = cache(), cache()
        ang = torch.arange(max_positions, device="cuda")[:, None] * 10000.0 ** (
            -torch.arange(0, DIM, 2, device="cuda", dtype=torch.float64) / DIM)
        self.cos_sin = torch.cat([ang.cos(), ang.sin()], 1).float()
        self.h = ar.ar_create(n, max_tokens * hidden * 2)
        self.cache = ar.ar_kv_create(self.h, self.k, self.v, "bf16", self.kv, DIM, PAGE, pages, self.kv * PAGE * DIM,
                                     PAGE * DIM, DIM)

    def close(self):
        ar.check(ar.ar_status(self.h), "a step")
        ar.check(ar.ar_kv_destroy(self.cache), "ar_kv_destroy")
        ar.check(ar.ar_destroy(self.h), "ar_destroy")

    def step(self, batch, y, residual, stream):
        """y: every rank's normed input [tokens][hidden]; returns the next normed input and residual."""
        T, row, out_row = batch.tokens, (self.q + 2 * self.kv) * DIM, self.q * DIM
        qkv = [a @ w for a, w in zip(y, self.w_qkv)]
        k, v = [x[:, out_row:] for x in qkv], [x[:, out_row + self.kv * DIM:] for x in qkv]
        q = [torch.empty((T, out_row), dtype=torch.bfloat16, device="cuda") for _ in range(self.n)]
        ar.check(ar.ar_rope_append(self.cache, batch, qkv, k, v, q, self.q, row, row, out_row, self.cos_sin,
                                   self.cos_sin.shape[0], DIM, 0, stream), "ar_rope_append")
        out = [torch.empty_like(x) for x in q]
        ar.check(ar.ar_paged_attention(self.cache, batch, q, out, self.q, out_row, out_row, DIM**-0.5, 0, stream),
                 "ar_paged_attention")
        parts = [o @ w for o, w in zip(out, self.w_o)]
        nxt = [torch.empty_like(p) for p in parts]
        ar.check(ar.ar_allreduce_block_norm(self.h, parts, residual, self.post, self.gate, 0, self.pre, 1.0, BETA, EPS,
                                            nxt, residual, T, self.hidden, "bf16", stream), "ar_allreduce_block_norm")
        return nxt, residual

    def plain(self, past, new, y, residual):
        """The same in fp64, one sequence after the other; `past`: each one's keys and values, which it extends."""
        d = lambda t: t.double()
        block = torch.zeros((sum(new), self.hidden), dtype=torch.float64, device="cuda")
        rms = lambda x: x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS)
        t = 0
        for s, q in enumerate(new):
            for r in range(self.n):
                x = (d(y[t: t + q]) @ d(self.w_qkv[r])).view(q, -1, DIM)
                have = past[s][r][0].shape[0]
                z = torch.complex(x[..., : DIM // 2].contiguous(), x[..., DIM // 2:].contiguous())
                turn = torch.complex(*d(self.cos_sin[have: have + q]).split(DIM // 2, 1))[:, None]
                z = torch.view_as_real(z * turn)
                x[:, : self.q + self.kv] = torch.cat([z[..., 0], z[..., 1]], -1)[:, : self.q + self.kv]
                k = torch.cat([past[s][r][0], x[:, self.q: self.q + self.kv]])
                v = torch.cat([past[s][r][1], x[:, self.q + self.kv:]])
                past[s][r] = (k, v)
                k, v = (a.repeat_interleave(self.q // self.kv, 1) for a in (k, v))
                p = torch.einsum("qhd,khd->hqk", x[:, : self.q], k) * DIM**-0.5
                hidden = torch.arange(have + q, device="cuda") > torch.arange(have, have + q, device="cuda")[:, None]
                p = torch.softmax(p.masked_fill(hidden, -math.inf), -1)
                block[t: t + q] += torch.einsum("hqk,khd->qhd", p, v).reshape(q, -1) @ d(self.w_o[r])
            t += q
        r = d(residual) + BETA * d(self.gate) * rms(block) * d(self.post)
        return rms(r) * d(self.pre), r


def main(argv=None):
    p = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    p.add_argument("--ranks", type=int, default=8)
    p.add_argument("--hidden", type=int, default=1024)
    p.add_argument("--steps", type=int, default=4)
    p.add_argument("--check", action="store_true")
    a = p.parse_args(argv)
    prompts = [70, 1, 200]
    length, width = [0] * len(prompts), -(-(max(prompts) + a.steps) // PAGE)
    layer = Layer(a.ranks, a.hidden, 4 * a.ranks, a.ranks, len(prompts) * width, sum(prompts), max(prompts) + a.steps)
    # pages are handed out in no order
    table = torch.randperm(len(prompts) * width, generator=torch.Generator().manual_seed(1)).int().view(-1, width).cuda()
    past = [[(torch.zeros((0, layer.kv, DIM), dtype=torch.float64, device="cuda"),) * 2 for _ in range(a.ranks)]
            for _ in prompts]
    g = torch.Generator(device="cuda").manual_seed(2)
    worst = 0.0
    for step in range(a.steps):
        new = prompts if step == 0 else [1] * len(prompts)      # the prompts, then one token each
        length = [x + q for x, q in zip(length, new)]
        start = torch.tensor([0] + new).cumsum(0).int().cuda()
        batch = ar.ar_batch(sum(new), len(new), max(new), start, kv_len := torch.tensor(length).int().cuda(), table, width)
        x = torch.randn((sum(new), a.hidden), generator=g, device="cuda").bfloat16()
        want = layer.plain(past, new, x, x) if a.check else None
        y, r = layer.step(batch, [x] * a.ranks, x.clone(), torch.cuda.current_stream())
        if a.check:
            err = [float((got.double() - w).norm() / w.norm()) for got, w in zip((y[-1], r), want)]
            worst = max(worst, *err)
            print(f"step {step}: {sum(new)} tokens, relative error {err[0]:.2e} of the output, {err[1]:.2e} of the residual")
        else:
            print(f"step {step}: {sum(new)} tokens, |y| {float(y[0].float().norm()):.4f}")
    layer.close()
    # bf16 rounds q, k, v, the attention's output, the parts and y: half a step, 2^-8, each at most
    return int(worst > 6 * 2.0**-8)


if __name__ == "__main__":
    sys.exit(main())
