"""Batches, paged caches and tolerances for the GPU tests of the layer's calls."""

from __future__ import annotations

import numpy as np
import torch

import all_reduce_reduction_rank_gb300 as ar

TORCH = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
HALF_STEP = {t: torch.finfo(d).eps / 2 for t, d in TORCH.items()}
TINY = {"f32": 0.0, "bf16": 0.0, "f16": 2.0**-25}      # half a step of the smallest fp16 numbers


def f64(t: torch.Tensor) -> np.ndarray:
    return t.detach().float().cpu().numpy().astype(np.float64)


class Layer:
    """n ranks' paged caches and one batch over them.  Slots that no call may
    use hold NaN, table entries that no call may read hold -1."""

    def __init__(self, n, kv_heads, dim, page, dtype, new, kv, *, seed=0, order="head", first_kept=None, spare=2,
                 max_new=None, pages=None, low=0):
        g = torch.Generator().manual_seed(seed)
        self.n, self.hk, self.dim, self.page, self.dtype, self.new, self.kv = n, kv_heads, dim, page, dtype, new, kv
        dt = TORCH[dtype]
        per = [-(-max(x, 0) // page) for x in kv]
        self.pages = pages or sum(per) + spare
        shape = (self.pages, page, kv_heads, dim) if order == "slot" else (self.pages, kv_heads, page, dim)
        nan = lambda *s: torch.full(s, float("nan"), dtype=dt, device="cuda")
        if order == "pair":     # keys and values of a page side by side in one allocation
            both = [nan(self.pages, 2, *shape[1:]) for _ in range(n)]
            self.k, self.v = [t[:, 0] for t in both], [t[:, 1] for t in both]
        else:
            self.k, self.v = [nan(*shape) for _ in range(n)], [nan(*shape) for _ in range(n)]
        st = self.k[0].stride()
        self.strides = (st[0], st[2], st[1]) if order == "slot" else (st[0], st[1], st[2])
        head = lambda c: c.transpose(1, 2) if order == "slot" else c    # [page, head, slot, dim] views
        self.kview, self.vview = [head(c) for c in self.k], [head(c) for c in self.v]
        ids = (torch.randperm(self.pages - low, generator=g) + low)[: sum(per)].tolist()
        self.width = max(1, max(per, default=1)) + 1
        table = torch.full((max(1, len(kv)), self.width), -1, dtype=torch.int32)
        self.keys = [[torch.randn((max(x, 0), kv_heads, dim), generator=g).to(dt) for x in kv] for _ in range(n)]
        self.vals = [[torch.randn((max(x, 0), kv_heads, dim), generator=g).to(dt) for x in kv] for _ in range(n)]
        at = 0
        for s, x in enumerate(kv):
            keep = 0 if first_kept is None else first_kept[s]       # keys before it are gone from the cache
            for j in range(per[s]):
                lo, hi = max(j * page, keep), min((j + 1) * page, x)
                if hi > lo:
                    table[s, j] = ids[at + j]
                    for r in range(n):
                        for c, src in ((self.kview[r], self.keys[r][s]), (self.vview[r], self.vals[r][s])):
                            c[ids[at + j], :, lo - j * page: hi - j * page] = src[lo:hi].transpose(0, 1).cuda()
            at += per[s]
        starts = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        self.starts, self.tokens = starts.tolist(), int(starts[-1])
        self.table, self.q_start = table.cuda(), torch.from_numpy(starts).cuda()
        self.kv_len = torch.tensor(kv, dtype=torch.int32).cuda()
        self.batch = ar.ar_batch(self.tokens, len(kv), max_new or max(1, max(new, default=1)), self.q_start,
                                 self.kv_len, self.table, self.width)
        self.gen = g

    def __enter__(self):
        self.h = ar.ar_create(self.n, 1 << 10)
        self.handle = ar.ar_kv_create(self.h, self.k, self.v, self.dtype, self.hk, self.dim, self.page, self.pages,
                                      *self.strides)
        return self

    def __exit__(self, *exc):
        assert ar.ar_kv_destroy(self.handle) == ar.AR_OK
        assert ar.ar_destroy(self.h) == ar.AR_OK
        return False

    def rows(self, heads, stride=None, fill=None):
        """[tokens][heads * dim] per rank inside rows of `stride` elements."""
        stride = stride or heads * self.dim
        out = []
        for _ in range(self.n):
            t = torch.full((self.tokens + 2, stride), float("nan"), dtype=TORCH[self.dtype])
            if fill != "nan":
                t[1:-1, : heads * self.dim] = torch.randn((self.tokens, heads * self.dim), generator=self.gen).to(t.dtype)
            out.append(t.cuda()[1:])
        return out
