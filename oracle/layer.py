"""Plain 64-bit definitions of the calls around the all-reduce in a layer --
TEST INFRASTRUCTURE ONLY: rotation and append to a paged cache, causal
attention of new tokens over it, and the norms around a block.

numpy float64, one sequence, token and head at a time where that is the
plainest; each function also returns the magnitude that its error bound
scales with.  Pinned by ``tests/test_oracle_layer.py``.
"""

from __future__ import annotations

import numpy as np


def rotate(x: np.ndarray, cos_sin_row: np.ndarray, interleaved: bool) -> tuple[np.ndarray, np.ndarray]:
    """One head x [D] turned by a table row [cos R/2, sin R/2]; and |x1 c| + |x2 s| per element."""
    x = x.astype(np.float64)
    R = cos_sin_row.shape[0]
    c, s = cos_sin_row[: R // 2].astype(np.float64), cos_sin_row[R // 2:].astype(np.float64)
    y, size = x.copy(), np.abs(x)
    i, j = (slice(0, R, 2), slice(1, R, 2)) if interleaved else (slice(0, R // 2), slice(R // 2, R))
    y[..., i] = x[..., i] * c - x[..., j] * s
    y[..., j] = x[..., j] * c + x[..., i] * s
    size[..., i] = np.abs(x[..., i] * c) + np.abs(x[..., j] * s)
    size[..., j] = np.abs(x[..., j] * c) + np.abs(x[..., i] * s)
    return y, size


def positions(q_start, kv_len):
    """(sequence, position) of every packed token."""
    out = []
    for s in range(len(kv_len)):
        new = q_start[s + 1] - q_start[s]
        out += [(s, kv_len[s] - new + i) for i in range(new)]
    return out


def attention(q: np.ndarray, k: np.ndarray, v: np.ndarray, first: int, scale: float, window: int):
    """q [new, heads, D] of one sequence whose first new token has position
    `first`; k, v [keys, kv heads, D].  Returns out and three magnitudes per
    element: sum p |v|, and per row the largest sum |q k| scale and |score|."""
    q, k, v = (a.astype(np.float64) for a in (q, k, v))
    new, heads, D = q.shape
    group = heads // k.shape[1]
    out, size = np.zeros_like(q), np.zeros_like(q)
    dots, top = np.zeros((new, heads, 1)), np.zeros((new, heads, 1))
    for i in range(new):
        pos = first + i
        lo = max(0, pos - window + 1) if window else 0
        if pos + 1 <= lo:
            continue
        for h in range(heads):
            kk, vv = k[lo: pos + 1, h // group], v[lo: pos + 1, h // group]
            s = kk @ q[i, h] * scale
            p = np.exp(s - s.max())
            p /= p.sum()
            out[i, h] = p @ vv
            size[i, h] = p @ np.abs(vv)
            dots[i, h] = (np.abs(kk) @ np.abs(q[i, h])).max() * scale
            top[i, h] = np.abs(s).max()
    return out, size, dots, top


def block_norm(xs, residual, post, gate, pre, alpha, beta, eps):
    """(y, r, |terms of r|); xs: the ranks' [tokens, hidden], post and gate may be None."""
    xs = [x.astype(np.float64) for x in xs]
    a, size = sum(xs), sum(np.abs(x) for x in xs)
    if post is not None:
        f = post.astype(np.float64) / np.sqrt((a * a).mean(-1, keepdims=True) + eps)
        a, size = a * f, size * np.abs(f)
    if gate is not None:
        a, size = a * gate.astype(np.float64), size * np.abs(gate.astype(np.float64))
    r = alpha * residual.astype(np.float64) + beta * a
    size = np.abs(alpha * residual.astype(np.float64)) + abs(beta) * size
    y = r / np.sqrt((r * r).mean(-1, keepdims=True) + eps) * pre.astype(np.float64)
    return y, r, size
