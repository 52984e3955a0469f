"""ar_paged_attention against the 64-bit definition: head groups, lengths from
none to thousands, ragged batches, windows, cache orders and strides, slots
and table entries that nothing may use, splits over CTAs, streams and graphs.

Tolerance, per element, u = half a step of the type, A = sum p |v|:
  u |out|                   the output's rounding
  u A                       the probabilities' rounding before they meet the values
  2 d A                     scores off by d <= D 2^-24 max sum|q k| scale + 2^-21 (|score| + 16): the fp32
                            dot product, the scaling, and ex2.approx (2^-22) over parts
  (keys + 64) 2^-24 2 A     the fp32 sums"""

import numpy as np
import pytest
import torch

import all_reduce_reduction_rank_gb300 as ar
from layer_util import HALF_STEP, TINY, TORCH, Layer, f64
from oracle import layer

pytestmark = pytest.mark.gpu


def expect(L, q, heads, scale, window, rank, s):
    a, b = L.starts[s], L.starts[s + 1]
    x = f64(q[rank][a:b, : heads * L.dim]).reshape(b - a, heads, L.dim)
    want, size, dots, top = layer.attention(x, f64(L.keys[rank][s]), f64(L.vals[rank][s]), L.kv[s] - (b - a), scale,
                                            window)
    u = HALF_STEP[L.dtype]
    d = L.dim * 2.0**-24 * dots + 2.0**-21 * (top + 16)
    tol = u * np.abs(want) + size * (u + 2 * d + 2 * (L.kv[s] + 64) * 2.0**-24) + TINY[L.dtype]
    return want, tol


def compare(L, q, out, heads, scale, window, seqs=None):
    for r in range(L.n):
        for s in range(len(L.kv)) if seqs is None else seqs:
            a, b = L.starts[s], L.starts[s + 1]
            if a == b:
                continue
            want, tol = expect(L, q, heads, scale, window, r, s)
            got = f64(out[r][a:b, : heads * L.dim]).reshape(want.shape)
            bad = ~(np.abs(got - want) <= tol)
            assert not bad.any(), (f"rank {r} sequence {s}: {bad.sum()} of {bad.size} off, first at "
                                   f"{np.argwhere(bad)[0]}: {got[bad][0]} for {want[bad][0]}")


def run(L, heads, *, window=0, scale=None, q_stride=None, out_stride=None, stream=None, q=None):
    scale = scale or L.dim**-0.5
    q = q or L.rows(heads, q_stride)
    out = L.rows(heads, out_stride, fill="nan")
    width = heads * L.dim
    rc = ar.ar_paged_attention(L.handle, L.batch, q, out, heads, q_stride or width, out_stride or width, scale, window,
                               stream)
    assert rc == ar.AR_OK
    assert ar.ar_status(L.h) == ar.AR_OK
    for t in out:   # nothing past the heads or the tokens is written
        assert torch.isnan(t[: L.tokens, width:].float()).all() and torch.isnan(t[L.tokens:].float()).all()
    return q, out


def check(n, kv_heads, group, dim, page, dtype, new, kv, *, window=0, seed=0, **k):
    strides = {x: k.pop(x) for x in ("q_stride", "out_stride") if x in k}
    first = None
    if window:
        first = [max(0, x - q - window + 1) for q, x in zip(new, kv)]
        first = [min(max(0, f), max(0, x)) for f, x in zip(first, kv)]
    with Layer(n, kv_heads, dim, page, dtype, new, kv, seed=seed, first_kept=first, **k) as L:
        q, out = run(L, kv_heads * group, window=window, **strides)
        compare(L, q, out, kv_heads * group, L.dim**-0.5, window)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("kv", [1, 15, 16, 17, 63, 64, 65, 127, 300])
def test_one_token(kv, dim, dtype):
    check(2, 1, 4, dim, 16, dtype, [1], [kv], seed=kv)


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("group", [1, 3, 5, 8, 16, 17, 40, 64])
def test_head_groups_and_pages(group, page):
    check(2, 2, group, 64 if page == 64 else 128, page, "bf16", [1, 1, 1], [77, 1, 200], seed=group)


@pytest.mark.parametrize("order", ["head", "slot"])
@pytest.mark.parametrize("dtype,dim", [("bf16", 128), ("f16", 64)])
def test_ragged_decodes(dtype, dim, order):
    new = [1, 0, 1, 2, 1, 4, 0, 3, 1]
    kv = [600, 5, 1, 2, 129, 700, 0, 3, 64]
    check(3, 2, 4, dim, 32, dtype, new, kv, order=order, q_stride=2 * 8 * dim + 8, out_stride=8 * dim + 16)


@pytest.mark.parametrize("new,kv", [([130], [130]), ([64, 1, 33], [64, 500, 40]), ([257, 3], [300, 3]),
                                    ([1, 200, 1], [333, 1000, 1]), ([128], [256]), ([513], [640])])
@pytest.mark.parametrize("dtype,dim,group", [("bf16", 128, 4), ("f16", 64, 3), ("bf16", 64, 1), ("f16", 128, 8)])
def test_chunks(new, kv, dtype, dim, group):
    check(2, 1, group, dim, 16, dtype, new, kv, seed=sum(kv))


@pytest.mark.parametrize("window", [1, 2, 16, 17, 100, 128, 129, 1000])
@pytest.mark.parametrize("new,kv", [([1, 1], [300, 90]), ([150, 1, 40], [500, 260, 40])])
def test_windows(window, new, kv):
    check(2, 1, 4, 128, 32, "bf16", new, kv, window=window, seed=window)


@pytest.mark.parametrize("max_new", [1, 500])
def test_the_widest_window_is_none(max_new):
    # also for rows before the first key, whose lower end would pass 32 bits
    new, kv = [9, 1], [4, 300]
    with Layer(2, 1, 64, 16, "f16", new, kv, max_new=max_new) as L:
        q, out = run(L, 3, window=2**31 - 1)
        compare(L, q, out, 3, L.dim**-0.5, 0)


@pytest.mark.parametrize("max_new", [1, 500])   # both kernels, whatever the batch is
def test_rows_that_see_nothing_are_zero(max_new):
    new, kv = [3, 2, 5, 1, 40], [1, 0, 5, 0, 7]
    with Layer(2, 1, 128, 16, "bf16", new, kv, max_new=max_new) as L:
        q, out = run(L, 4)
        compare(L, q, out, 4, L.dim**-0.5, 0)
        for r in range(2):
            assert (out[r][:2] == 0).all() and (out[r][3:5] == 0).all() and (out[r][10] == 0).all()


@pytest.mark.parametrize("max_new", [1, 500])
@pytest.mark.parametrize("new,kv", [([1, 1, 1], [40, 1000, 129]), ([70, 1, 9], [200, 300, 9])])
def test_either_kernel_gives_the_definition(max_new, new, kv):
    check(2, 2, 5, 128, 64, "f16", new, kv, max_new=max_new)


@pytest.mark.parametrize("max_new", [1, 500])
def test_keys_and_values_in_one_allocation(max_new):
    check(2, 3, 4, 64, 32, "bf16", [1, 30, 2], [100, 45, 64], order="pair", max_new=max_new)


@pytest.mark.parametrize("seed", range(12))
@pytest.mark.parametrize("max_new", [1, 500])
def test_random_batches(seed, max_new):
    rng = np.random.default_rng(seed)
    pick = lambda *xs: xs[int(rng.integers(len(xs)))]
    seqs = int(rng.integers(1, 12))
    new = [int(x) for x in rng.integers(0, pick(3, 40, 150), seqs)]
    kv = [max(0, int(q + x - pick(0, 0, 3))) for q, x in zip(new, rng.integers(0, pick(5, 300, 900), seqs))]
    if sum(new) == 0:
        new[0], kv[0] = 1, kv[0] + 1
    check(int(rng.integers(2, 5)), pick(1, 2), pick(1, 2, 4, 6, 7), pick(64, 128), pick(16, 32, 64, 128),
          pick("bf16", "f16"), new, kv, window=pick(0, 0, int(rng.integers(1, 200))), order=pick("head", "slot", "pair"),
          max_new=max_new, seed=seed)


@pytest.mark.parametrize("max_new", [1, 500])
def test_chains_without_programmatic_launch(max_new):
    with Layer(2, 1, 128, 16, "bf16", [1, 50], [700, 90], max_new=max_new) as L:
        assert ar.ar_set_option(L.h, ar.AR_OPT_PDL, 0) == ar.AR_OK
        q, out = run(L, 4)
        compare(L, q, out, 4, L.dim**-0.5, 0)
        with_pdl = [o.clone() for o in out]
        assert ar.ar_set_option(L.h, ar.AR_OPT_PDL, 1) == ar.AR_OK
        for _ in range(5):   # back to back: each call finds the last one's workspace in use or free
            ar.check(ar.ar_paged_attention(L.handle, L.batch, q, out, 4, 512, 512, L.dim**-0.5, 0))
        assert ar.ar_status(L.h) == ar.AR_OK
        for x, y in zip(out, with_pdl):
            assert torch.equal(x[: L.tokens], y[: L.tokens])


def test_many_sequences():
    rng = np.random.default_rng(5)
    new = [int(x) for x in rng.integers(0, 3, 400)]
    kv = [int(max(q, x)) for q, x in zip(new, rng.integers(0, 90, 400))]
    check(2, 1, 4, 64, 16, "bf16", new, kv)


@pytest.mark.parametrize("max_new", [1, 500])
@pytest.mark.parametrize("dim", [64, 128])
def test_long_rows_are_split_and_joined_the_same_way_every_time(dim, max_new):
    # one sequence's keys over many CTAs; three runs in a row leave the joins' counters ready for the next
    with Layer(2, 1, dim, 128, "bf16", [2, 1], [20000, 3333], max_new=max_new) as L:
        q, out = run(L, 3)
        compare(L, q, out, 3, L.dim**-0.5, 0)
        for _ in range(2):
            _, again = run(L, 3, q=q)
            for x, y in zip(out, again):
                assert torch.equal(x[: L.tokens], y[: L.tokens])


@pytest.mark.parametrize("max_new", [1, 500])
def test_large_scores(max_new):
    # probabilities that are all but one-hot, and a reference that moves by hundreds
    with Layer(2, 1, 128, 16, "bf16", [3, 33], [150, 400], max_new=max_new) as L:
        q, out = run(L, 4, scale=2.0)
        compare(L, q, out, 4, 2.0, 0)


@pytest.mark.parametrize("max_new", [1, 500])
def test_infinite_scores_hide_their_keys(max_new):
    # a key whose scores are -inf for every row counts as hidden
    with Layer(2, 1, 64, 16, "bf16", [2], [50], max_new=max_new) as L:
        q = [t.abs().add_(0.1) for t in L.rows(2)]
        for r in range(2):
            page = int(L.table[0, 0])
            L.kview[r][page, 0, 7] = -float("inf")
            L.keys[r][0][7] = -30000.0   # in the definition: a score so low that its weight is 0
        out = L.rows(2, fill="nan")
        assert ar.ar_paged_attention(L.handle, L.batch, q, out, 2, 128, 128, 1.0, 0) == ar.AR_OK
        assert ar.ar_status(L.h) == ar.AR_OK
        for r in range(2):
            want, tol = expect(L, q, 2, 1.0, 0, r, 0)
            keys = [i for i in range(50) if i != 7]
            x = f64(q[r][:2, :128]).reshape(2, 2, 64)
            dots = np.abs(f64(L.keys[r][0])[keys, 0]).sum(-1).max() * np.abs(x).max()
            tol = HALF_STEP["bf16"] * np.abs(want) + np.abs(f64(L.vals[r][0])).max() * (
                HALF_STEP["bf16"] + 2 * (64 * 2.0**-24 + 2.0**-21) * (dots + 16) + 2.0**-16)
            got = f64(out[r][:2, :128]).reshape(want.shape)
            assert (np.abs(got - want) <= tol).all()


@pytest.mark.parametrize("max_new", [1, 500])
def test_cache_offsets_past_32_bits(max_new):
    # pages whose element offsets pass 2^31
    n, D, P = 2, 128, 128
    pages = (1 << 31) // (P * D) + 200
    free, _ = torch.cuda.mem_get_info()
    if free < 24 << 30:
        pytest.skip("needs 24 GB")
    with Layer(n, 1, D, P, "bf16", [1, 20], [500, 1000], pages=pages, low=pages - 150, max_new=max_new) as L:
        q, out = run(L, 4)
        compare(L, q, out, 4, L.dim**-0.5, 0)


@pytest.mark.parametrize("max_new", [1, 500])
def test_bad_entries_reach_no_memory_and_are_reported(max_new):
    def case(spoil, good):
        with Layer(2, 1, 64, 16, "bf16", [1, 1, 20], [50, 70, 40], max_new=max_new) as L:
            spoil(L)
            q, out = L.rows(4), L.rows(4, fill="nan")
            assert ar.ar_paged_attention(L.handle, L.batch, q, out, 4, 256, 256, 0.125, 0) == ar.AR_OK
            assert ar.ar_status(L.h) == ar.AR_ERR_INDEX
            assert ar.ar_status(L.h) == ar.AR_OK
            compare(L, q, out, 4, 0.125, 0, good)
            for t in out:
                assert torch.isnan(t[L.tokens:].float()).all()

    case(lambda L: L.table[1].fill_(L.pages), [0, 2])
    case(lambda L: L.table[1].fill_(-7), [0, 2])
    case(lambda L: L.kv_len[0:1].fill_(-1), [1, 2])
    case(lambda L: L.kv_len[0:1].fill_(1 << 30), [1, 2])
    case(lambda L: L.q_start[3:4].fill_(23), [0, 1])
    case(lambda L: L.q_start[3:4].fill_(1), [0, 1])


@pytest.mark.parametrize("max_new", [1, 500])
def test_another_stream_and_graph_replay_with_other_lengths(max_new):
    with Layer(2, 1, 128, 16, "bf16", [1, 40], [100, 200], max_new=max_new) as L:
        q, out = L.rows(4), L.rows(4, fill="nan")
        call = lambda s: ar.check(ar.ar_paged_attention(L.handle, L.batch, q, out, 4, 512, 512, 0.1, 0, s))
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            call(s)
        s.synchronize()
        compare(L, q, out, 4, 0.1, 0)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            call(s)
        for kv in ([100, 200], [37, 41], [99, 160]):
            L.kv_len.copy_(torch.tensor(kv, dtype=torch.int32))
            L.kv = kv
            keep = [[t[:x] for t, x in zip(ks, kv)] for ks in L.keys], [[t[:x] for t, x in zip(vs, kv)] for vs in L.vals]
            full = L.keys, L.vals
            L.keys, L.vals = keep
            for t in out:
                t[: L.tokens].fill_(float("nan"))
            g.replay()
            torch.cuda.synchronize()
            assert ar.ar_status(L.h) == ar.AR_OK
            compare(L, q, out, 4, 0.1, 0)
            L.keys, L.vals = full


def test_no_tokens_is_a_no_op_and_handles_are_checked():
    with Layer(2, 1, 64, 16, "bf16", [0, 0], [5, 0]) as L:
        q = [torch.zeros(64, dtype=TORCH["bf16"], device="cuda") for _ in range(2)]
        out = [torch.ones(64, dtype=TORCH["bf16"], device="cuda") for _ in range(2)]
        assert ar.ar_paged_attention(L.handle, L.batch, q, out, 1, 64, 64, 0.1, 0) == ar.AR_OK
        assert ar.ar_traffic(L.h).launches == 0
        assert all((t == 1).all() for t in out)
        assert ar.ar_paged_attention(None, L.batch, q, out, 1, 64, 64, 0.1, 0) == ar.AR_ERR_INVALID
        assert ar.ar_kv_destroy(None) == ar.AR_ERR_INVALID
