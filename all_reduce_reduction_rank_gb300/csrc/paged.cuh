// Device helpers of the paged-cache kernels: a sequence's place in the batch,
// the split of a call's key tiles over the CTAs, tensor copies of pages, and
// bounded waits.
#pragma once

#include <cmath>
#include <type_traits>

#include "bulk.cuh"
#include "common.cuh"
#include "layer.h"

namespace argb {

__device__ __forceinline__ void report_index(DevStatus* st) { atomicCAS(&st->code, 0, AR_ERR_INDEX); }

// One sequence of the batch: its first packed row, its new tokens, its keys
// and the position of its first new token (negative when it has fewer keys
// than new tokens).
struct Seq {
    int q0, nq, len, c0;
};

struct RawSeq {
    int q0, q1, len;
};

__device__ __forceinline__ RawSeq read_seq(const BatchArgs& b, int s)
{
    return RawSeq{b.q_start[s], b.q_start[s + 1], b.kv_len[s]};
}

// Values out of range reach no memory: a bad token range counts as no tokens,
// a bad length as no keys.
__device__ __forceinline__ Seq check_seq(const BatchArgs& b, const RawSeq& x, DevStatus* st)
{
    Seq r{x.q0, x.q1 - x.q0, x.len, 0};
    if (x.q0 < 0 || x.q1 < x.q0 || x.q1 > b.tokens) {
        report_index(st);
        r.q0 = r.nq = 0;
    }
    if (x.len < 0 || x.len > (1 << 30) || (size_t)x.len > (b.table_stride << b.page_shift)) {
        report_index(st);
        r.len = 0;
    }
    r.c0 = r.len - r.nq;
    return r;
}

// With masks of the call's own: the prefix too.
struct MaskedSeq : Seq {
    int prefix;                      // at most its keys
};

struct MaskedRawSeq : RawSeq {
    int prefix;
};

__device__ __forceinline__ MaskedRawSeq read_seq(const MaskedBatchArgs& b, int s)
{
    MaskedRawSeq x;
    static_cast<RawSeq&>(x) = read_seq(static_cast<const BatchArgs&>(b), s);
    x.prefix = b.prefix ? b.prefix[s] : 0;
    return x;
}

__device__ __forceinline__ MaskedSeq check_seq(const MaskedBatchArgs& b, const MaskedRawSeq& x, DevStatus* st)
{
    MaskedSeq r;
    static_cast<Seq&>(r) = check_seq(static_cast<const BatchArgs&>(b), static_cast<const RawSeq&>(x), st);
    r.prefix = min(x.prefix, r.len);
    return r;
}

template <typename B>
__device__ __forceinline__ auto load_seq(const B& b, int s, DevStatus* st)
{
    return check_seq(b, read_seq(b, s), st);
}

// What a kernel knows of a sequence, by the batch it has.
template <typename B> struct SeqOf { using Raw = RawSeq; using Type = Seq; };
template <> struct SeqOf<MaskedBatchArgs> { using Raw = MaskedRawSeq; using Type = MaskedSeq; };

// Another lane's sequence.
__device__ __forceinline__ Seq shfl_seq(const Seq& q, int src)
{
    return Seq{__shfl_sync(0xffffffffu, q.q0, src), __shfl_sync(0xffffffffu, q.nq, src),
               __shfl_sync(0xffffffffu, q.len, src), __shfl_sync(0xffffffffu, q.c0, src)};
}

__device__ __forceinline__ MaskedSeq shfl_seq(const MaskedSeq& q, int src)
{
    MaskedSeq r;
    static_cast<Seq&>(r) = shfl_seq(static_cast<const Seq&>(q), src);
    r.prefix = __shfl_sync(0xffffffffu, q.prefix, src);
    return r;
}

// Keys of a token at position p end before this: what the causal mask shows (also
// of the last of several tokens), and the prefix.
__host__ __device__ __forceinline__ int seen_end(const Seq&, int causal_end) { return causal_end > 0 ? causal_end : 0; }
__host__ __device__ __forceinline__ int seen_end(const MaskedSeq& q, int causal_end)
{
    return causal_end > 0 ? max(causal_end, q.prefix) : 0;
}

// The sequence of token t: the last s with q_start[s] <= t.  A warp looks at
// 32 places of the range at once.
__device__ __forceinline__ int seq_of(const int32_t* q_start, int seqs, int t, int lane)
{
    int lo = 0, hi = seqs;   // q_start[lo] <= t, answer in [lo, hi)
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) / 32;
        const int at = lo + lane * step;
        const bool below = at < hi && q_start[at] <= t;
        const int k = 31 - __clz(__ballot_sync(0xffffffffu, below) | 1u);
        const int nlo = lo + k * step;
        hi = min(hi, nlo + step);
        lo = nlo;
    }
    return lo;
}

// ---- split of the work ------------------------------------------------------------
// A row tile is TM consecutive new tokens of a sequence with the query heads of
// one head group; it costs one unit per tile of KT keys between the first key
// any of its rows sees and the last (at least one, so that rows that see
// nothing are written too), and W units for its start and end.  The units of
// all (head group, sequence, row tile) triples, in that order, are cut into
// equal runs, one per CTA, whatever the lengths are.  A cut that falls within
// an eighth of a run (W to SNAP units) of a triple's edge moves to that edge: the
// triples that stay cut are joined afterwards, which costs more than that
// imbalance.  Only the first
// and the last triple of a run can be shared with other CTAs.

template <int KT_, int W_, int SNAP_>
struct Split {
    static constexpr int KT = KT_, W = W_, SNAP = SNAP_;
    static_assert(SNAP >= W, "a cut that stays lies among the key tiles");
};

struct Span {
    int key_lo, key_hi;   // keys that some row of the tile sees (key_hi <= key_lo: none)
    int j_lo, tiles;      // first key tile, number of tiles (>= 1)
};

template <int KT>
__host__ __device__ __forceinline__ Span span_of(const Seq& q, int tm, int t, int window)
{
    const int first = q.c0 + t * tm;                                // position of the tile's first token
    const int end = (t + 1) * tm, last = q.c0 + (end < q.nq ? end : q.nq);   // one past its last token's position
    Span p;
    p.key_hi = last > 0 ? last : 0;
    p.key_lo = window > 0 && first - window + 1 > 0 ? first - window + 1 : 0;
    p.j_lo = p.key_lo / KT;
    const int tiles = (p.key_hi + KT - 1) / KT - p.j_lo;
    p.tiles = tiles > 1 ? tiles : 1;
    return p;
}

// A row tile's span in the batch; the first keys of its tokens never decrease.
template <int KT>
__host__ __device__ __forceinline__ Span tile_span(const BatchArgs& b, const Seq& q, int tm, int t)
{
    return span_of<KT>(q, tm, t, b.window);
}

template <int KT>
__host__ __device__ __forceinline__ Span tile_span(const MaskedBatchArgs& b, const MaskedSeq& q, int tm, int t)
{
    Span p = span_of<KT>(q, tm, t, b.window);
    p.key_hi = seen_end(q, p.key_hi);
    if (b.first) p.key_lo = max(p.key_lo, b.first[q.q0 + t * tm]);
    p.key_lo = min(p.key_lo, p.key_hi);
    p.j_lo = p.key_lo / KT;
    p.tiles = max((p.key_hi + KT - 1) / KT - p.j_lo, 1);
    return p;
}

typedef unsigned long long u64;

// Units of all row tiles of a sequence; a long prompt has more than 2^32 (a million
// tokens, one to a row tile, 64 keys to a key tile: 2^33).
template <typename S>
__host__ __device__ __forceinline__ u64 units_of_sequence(const Seq& q, int tm, int window)
{
    u64 sum = 0;
    const int nt = (q.nq + tm - 1) / tm;
    for (int t = 0; t < nt; ++t) sum += (u64)(span_of<S::KT>(q, tm, t, window).tiles + S::W);
    return sum;
}

template <typename S>
__host__ __device__ __forceinline__ u64 units_in(const BatchArgs& b, const Seq& q, int tm)
{
    return units_of_sequence<S>(q, tm, b.window);
}

template <typename S>
__host__ __device__ __forceinline__ u64 units_in(const MaskedBatchArgs& b, const MaskedSeq& q, int tm)
{
    u64 sum = 0;
    const int nt = (q.nq + tm - 1) / tm;
    for (int t = 0; t < nt; ++t) sum += (u64)(tile_span<S::KT>(b, q, tm, t).tiles + S::W);
    return sum;
}

struct Cursor {
    u64 begin;                   // first unit of the current triple
    u64 end;                     // where the next CTA's run begins, before it is moved to an edge
    u64 total;                   // units of the call
    unsigned ctas;               // CTAs that share them
    int snap;                    // an eighth of a run, W to SNAP
    int head, s, t;              // the current triple
    int tile;                    // its first key tile of this CTA
};

// a / b; most calls are small enough for the 32-bit division, a fraction of the other's time
__device__ __forceinline__ u64 quotient(u64 a, u64 b)
{
    return ((a | b) >> 32) == 0 ? (u64)((unsigned)a / (unsigned)b) : a / b;
}

__device__ __forceinline__ u64 run_begin(u64 total, unsigned ctas, unsigned c) { return quotient(total * c, ctas); }

// The last CTA whose run begins at or before unit u.
__device__ __forceinline__ unsigned cta_of(u64 total, unsigned ctas, u64 u)
{
    return (unsigned)quotient((u + 1) * ctas - 1, total);
}

struct SplitShared {
    u64 warp_sum[32];
    u64 off;
    int s;
};

// Where a run begins, from the units before its triple's sequence (`off`: the
// run's first unit within that sequence).  Every warp walks the sequence's row
// tiles, 32 at a time.
template <typename S, typename B, typename Q>
__device__ __forceinline__ void enter_sequence(const B& b, int tm, const Q& q, u64 g, u64 off, Cursor& c)
{
    const int lane = threadIdx.x & 31;
    auto units_of = [&](int t) { return (unsigned)(tile_span<S::KT>(b, q, tm, t).tiles + S::W); };
    const int nt = (q.nq + tm - 1) / tm;
    c.t = 0;
    for (int t0 = 0; nt > 1; t0 += 32) {
        const int t = t0 + lane;
        const u64 u = t < nt ? units_of(t) : 0;
        u64 in = u;
        for (int o = 1; o < 32; o <<= 1) {
            const u64 x = __shfl_up_sync(0xffffffffu, in, o);
            if (lane >= o) in += x;
        }
        const unsigned here = __ballot_sync(0xffffffffu, in > off);
        if (here) {
            const int src = __ffs(here) - 1;
            c.t = t0 + src;
            off -= __shfl_sync(0xffffffffu, in - u, src);
            break;
        }
        if (t0 + 32 >= nt) break;   // not reached: the tiles' units cover `off`
        off -= __shfl_sync(0xffffffffu, in, 31);
    }
    c.begin = g - off;
    const int units = (int)units_of(c.t), o = (int)off, snap = min(c.snap, units / 2);
    c.tile = o <= snap ? 0 : units - o <= snap ? units - S::W : o - S::W;
}

// The runs, from the units of one head group; false for a CTA without one.
template <typename S>
__device__ __forceinline__ bool cut_runs(u64 per_head, int heads, int min_units, Cursor& c, u64& g, u64& in_head)
{
    c.total = per_head * (unsigned)heads;
    c.ctas = gridDim.x;
    const u64 most = quotient(c.total + min_units - 1, min_units);
    if (most < c.ctas) c.ctas = (unsigned)most;
    if (blockIdx.x >= c.ctas) return false;
    g = run_begin(c.total, c.ctas, blockIdx.x);
    c.end = run_begin(c.total, c.ctas, blockIdx.x + 1);
    if (S::SNAP > 0) {
        const u64 eighth = quotient(c.total, c.ctas) / 8;
        c.snap = eighth < (u64)S::W ? S::W : eighth > (u64)S::SNAP ? S::SNAP : (int)eighth;
    } else {
        c.snap = 0;
    }
    c.head = (int)quotient(g, per_head);
    in_head = g - c.head * per_head;
    return true;
}

// split_work for at most 256 sequences of few row tiles each (decode steps):
// every warp goes over all of them by itself, without shared memory, barriers
// and second loads (1.9 us of a decode step's 10 went into the other form).
template <typename S, typename B>
__device__ bool split_few(const B& b, int tm, int heads, int min_units, Cursor& c, typename SeqOf<B>::Type& at,
                          DevStatus* st)
{
    const int lane = threadIdx.x & 31;
    const int per = (b.seqs + 31) / 32, s0 = min(lane * per, b.seqs), s1 = min(s0 + per, b.seqs);
    u64 mine = 0;
    typename SeqOf<B>::Type q{};
    if (per == 1) {
        if (s0 < s1) {
            q = load_seq(b, s0, st);
            mine = units_in<S>(b, q, tm);
        }
    } else {
        typename SeqOf<B>::Raw raw[8];   // all loads before the first use: a report orders what follows it
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (s0 + k < s1) raw[k] = read_seq(b, s0 + k);
#pragma unroll 1
        for (int k = 0; k < per; ++k) {
            if (s0 + k < s1) mine += units_in<S>(b, check_seq(b, raw[0], st), tm);
#pragma unroll
            for (int i = 0; i < 7; ++i) raw[i] = raw[i + 1];
        }
    }
    u64 incl = mine;
    for (int o = 1; o < 32; o <<= 1) {
        const u64 x = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += x;
    }
    u64 g, in_head;
    if (!cut_runs<S>(__shfl_sync(0xffffffffu, incl, 31), heads, min_units, c, g, in_head)) return false;
    const int src = __ffs(__ballot_sync(0xffffffffu, in_head < incl)) - 1;
    u64 off = in_head - (incl - mine);   // of lane src; the others' is not used
    int s = s0;
    if (per > 1 && lane == src)
        for (;; ++s) {
            q = load_seq(b, s, st);
            const u64 u = units_in<S>(b, q, tm);
            if (off < u) break;
            off -= u;
        }
    c.s = __shfl_sync(0xffffffffu, s, src);
    off = __shfl_sync(0xffffffffu, off, src);
    at = shfl_seq(q, src);
    enter_sequence<S>(b, tm, at, g, off, c);
    return true;
}

// Called by all NT threads; false for a CTA with nothing to do.  `min_units`:
// a run is at least that long, so that small calls do not pay for joins.  `at`:
// the sequence the run begins in.
template <typename S, int NT, typename B>
__device__ bool split_work(const B& b, int tm, int heads, int min_units, SplitShared* sh, Cursor& c,
                           typename SeqOf<B>::Type& at, DevStatus* st)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    // consecutive sequences for a warp's lanes; few sequences are spread over the warps
    const int of_warp = (b.seqs + NT / 32 - 1) / (NT / 32), per = (of_warp + 31) / 32;
    const int w0 = min(warp * of_warp, b.seqs), w1 = min(w0 + of_warp, b.seqs);
    const int s0 = min(w0 + lane * per, w1), s1 = min(s0 + per, w1);
    using Q = typename SeqOf<B>::Type;
    auto units_of = [&](const Q& q, int t) { return (unsigned)(tile_span<S::KT>(b, q, tm, t).tiles + S::W); };
    u64 mine = 0;
    // long sequences' row tiles are counted by the whole warp
    for (int k = 0; k < per; ++k) {
        const int s = s0 + k;
        Q q{};
        if (s < s1) q = load_seq(b, s, st);
        const int nt = (q.nq + tm - 1) / tm;
        const bool is_long = nt > 8;
        if (!is_long) mine += units_in<S>(b, q, tm);
        unsigned todo = __ballot_sync(0xffffffffu, is_long);
        while (todo) {
            const int src = __ffs(todo) - 1;
            todo &= todo - 1;
            const Q w = shfl_seq(q, src);
            const int wt = (w.nq + tm - 1) / tm;
            u64 sum = 0;
            for (int t = lane; t < wt; t += 32) sum += units_of(w, t);
            for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            if (lane == src) mine += sum;
        }
    }
    u64 incl = mine;
    for (int o = 1; o < 32; o <<= 1) {
        const u64 x = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += x;
    }
    if (lane == 31) sh->warp_sum[warp] = incl;
    __syncthreads();
    u64 before = 0, per_head = 0;
#pragma unroll
    for (int w = 0; w < NT / 32; ++w) {
        if (w < warp) before += sh->warp_sum[w];
        per_head += sh->warp_sum[w];
    }
    u64 g, in_head;
    if (!cut_runs<S>(per_head, heads, min_units, c, g, in_head)) return false;   // the whole CTA
    const u64 excl = before + incl - mine;
    if (in_head >= excl && in_head < excl + mine) {   // (false without sequences: mine is 0)
        // this thread's sequences hold it
        u64 at = excl;
        for (int s = s0; s < s1; ++s) {
            u64 sum = 0;
            if (s + 1 < s1) sum = units_in<S>(b, load_seq(b, s, st), tm);
            if (s + 1 == s1 || in_head < at + sum) {
                sh->s = s;
                sh->off = in_head - at;
                break;
            }
            at += sum;
        }
    }
    __syncthreads();
    c.s = sh->s;
    at = load_seq(b, c.s, st);
    enter_sequence<S>(b, tm, at, g, sh->off, c);
    return true;
}

// One triple's part in this CTA's run.
template <typename B>
struct Segment {
    typename SeqOf<B>::Type q;
    Span span;
    int head, s, t;
    int j0, j1;                       // key tiles of this CTA
    unsigned first_cta, parts, slot;  // CTA of its first part, its parts (1: whole), this CTA's partial slot
};

// Walks a run.  Every warp keeps its own copy; all read the same values.
template <typename S, typename B>
struct Walk {
    using Q = typename SeqOf<B>::Type;
    Cursor c;
    Q q;
    int loaded;

    Walk() = default;   // in shared memory
    __device__ __forceinline__ Walk(const Cursor& cur, const Q& at) : c(cur), q(at), loaded(cur.s) {}

    __device__ __forceinline__ bool next(const B& b, int tm, Segment<B>& seg, DevStatus* st)
    {
        for (;;) {
            if (c.begin >= c.end) return false;
            if (loaded != c.s) {
                q = load_seq(b, c.s, st);
                loaded = c.s;
            }
            if (c.t * tm >= q.nq) {
                c.t = 0;
                if (++c.s == b.seqs) {
                    c.s = 0;
                    ++c.head;
                }
                continue;
            }
            seg.span = tile_span<S::KT>(b, q, tm, c.t);
            const int units = seg.span.tiles + S::W, snap = min(c.snap, units / 2);
            const u64 left = c.end - c.begin;
            int stop = seg.span.tiles;   // one past this CTA's last tile
            bool last = false;
            if (left < (u64)units) {
                const int o = (int)left;
                last = true;
                if (o <= snap) return false;
                if (units - o > snap) stop = o - S::W;
            }
            const int start = c.tile;
            seg.first_cta = 0;
            seg.parts = 1;
            seg.slot = 0;
            if (start > 0 || stop < seg.span.tiles) {
                seg.first_cta = cta_of(c.total, c.ctas, c.begin + snap);
                seg.parts = cta_of(c.total, c.ctas, c.begin + units - snap - 1) - seg.first_cta + 1;
                seg.slot = 2 * blockIdx.x + (seg.first_cta == blockIdx.x ? 1 : 0);
            }
            seg.q = q;
            seg.head = c.head;
            seg.s = c.s;
            seg.t = c.t;
            seg.j0 = seg.span.j_lo + start;
            seg.j1 = seg.span.j_lo + stop;
            c.begin = last ? c.end : c.begin + units;
            c.tile = 0;
            ++c.t;
            if (start < stop) return true;   // else the run's first cut moved to the end of this triple
        }
    }
};

// Partial slot of part i of a triple whose first part is CTA f's.
__device__ __forceinline__ unsigned part_slot(unsigned f, unsigned i) { return i == 0 ? 2 * f + 1 : 2 * (f + i); }

// ---- copies, waits, arithmetic -------------------------------------------------------

// One box of a page: 64 elements by the map's tokens, at (d, slot, head, page).
__device__ __forceinline__ void page_copy(void* smem_dst, const CUtensorMap* map, int d, int slot, int head, int page,
                                          uint64_t* bar)
{
    asm volatile("cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
                 "[%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(smem_addr(smem_dst)),
                 "l"(map), "r"(d), "r"(slot), "r"(head), "r"(page), "r"(smem_addr(bar))
                 : "memory");
}

// One box of a packed [token][head][d] tensor.
__device__ __forceinline__ void box_copy(void* smem_dst, const CUtensorMap* map, int d, int head, int token,
                                         uint64_t* bar)
{
    asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
                 "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_addr(smem_dst)),
                 "l"(map), "r"(d), "r"(head), "r"(token), "r"(smem_addr(bar))
                 : "memory");
}

__device__ __forceinline__ void prefetch_map(const CUtensorMap* map)
{
    asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}

__device__ __forceinline__ void mbar_arrive(uint64_t* bar)
{
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}

__device__ __forceinline__ void fence_proxy_async()
{
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// pdl_acquire for kernels whose tensor copies read what the launch before wrote
// with ordinary stores (the queries, the caches' new slots).
__device__ __forceinline__ void pdl_acquire_for_copies()
{
    pdl_acquire();
    asm volatile("fence.proxy.async.global;" ::: "memory");
}

// Waits in the hardware, for about 20 us at most: a warp that polls takes issue
// slots from the warps of its scheduler that compute.
__device__ __forceinline__ bool mbar_wait_20us(uint64_t* bar, uint32_t parity)
{
    uint32_t done;
    asm volatile("{\n\t.reg .pred p;\n\t"
                 "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
                 "selp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(done)
                 : "r"(smem_addr(bar)), "r"(parity), "r"(20000u)
                 : "memory");
    return done != 0;
}

// Bounded wait: false after about a second (or once `stop` is set).
__device__ __forceinline__ bool wait_a_second(uint64_t* bar, uint32_t parity, volatile int* stop)
{
    const uint64_t t0 = globaltimer_ns();
#pragma unroll 1
    for (uint32_t i = 0; i < kMbarMaxPolls; ++i) {
        if (mbar_wait_20us(bar, parity)) return true;
        if ((stop && *stop) || globaltimer_ns() - t0 > 1000000000ull) return false;
    }
    return false;
}

// The same for the warps of a CTA that depend on one another, after a first
// mbar_wait_20us, the usual end: it also ends once another warp has given up, and
// giving up sets the status word.
__device__ __forceinline__ bool wait_on_or_give_up(uint64_t* bar, uint32_t parity, volatile int* gave_up, DevStatus* st)
{
    if (wait_a_second(bar, parity, gave_up)) return true;
    *gave_up = 1;
    report_wait_timeout(st);
    return false;
}

__device__ __forceinline__ bool wait_or_give_up(uint64_t* bar, uint32_t parity, volatile int* gave_up, DevStatus* st)
{
    return mbar_wait_20us(bar, parity) || wait_on_or_give_up(bar, parity, gave_up, st);
}

// Before a CTA ends, whoever issued asynchronous work of it waits for that work,
// however the CTA's other waits ended: what is in flight still writes this CTA's
// shared memory, which another CTA would own by then.
__device__ __forceinline__ void wait_for_own(uint64_t* bar, uint32_t parity, DevStatus* st)
{
    if (!wait_a_second(bar, parity, nullptr)) report_wait_timeout(st);
}

// wait_for_own for a ring of `stages` that `issued` tiles went through; `stage` and
// `phase` are the next tile's.  Usually the last tiles have long been waited for.
__device__ __forceinline__ void wait_for_ring(uint64_t* full, int stages, uint32_t issued, int stage, uint32_t phase,
                                              DevStatus* st)
{
#pragma unroll 1
    for (uint32_t k = 0; k < issued && k < (uint32_t)stages; ++k) {
        if (--stage < 0) {
            stage = stages - 1;
            phase ^= 1;
        }
        wait_for_own(&full[stage], phase, st);
    }
}

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// The softmax's probabilities are p = 2^(x - m), x the scores in base 2, against a
// reference m that is put kBelow under a row's maximum and moves only when one
// passes it by kBelow + kSlack: the accumulators are seldom rescaled, and p stays
// under 2^(kBelow + kSlack).  As the second product's operand p has the cache's type.
// bf16 reaches as far down as fp32.  fp16 ends at 2^-24 (and has a fixed step of that
// below 2^-14), but goes up to 2^16, so there the largest p is near 2^7 to 2^15 and not
// 1: what is lost of a probability is at most 2^-32 of the largest.
constexpr float kSlack = 8.0f;
template <int DT> constexpr float kBelow = DT == AR_F16 ? 7.0f : 0.0f;

// The first key of new token `tok`, which is not before that of `tile_tok`, the first
// token of its row tile: the tile's keys begin there.
__device__ __forceinline__ int first_key(const MaskedBatchArgs& b, const Seq& q, int tile_tok, int tok, DevStatus* st)
{
    const int f = b.first[q.q0 + tok];
    if (f < b.first[q.q0 + tile_tok]) report_index(st);
    return f;
}

// Magnitudes, in base 2, up to which the chunk kernel takes a capped score's bound for the maximum; with a bias.
constexpr double kBound = 30.0, kBiasedBound = 15.0;

// What becomes of a score s = q . k, in base 2: s scale_log2; or cap_log2 tanh(s to_cap); then
// less slope |distance|.
struct ScoreArgs {
    float cap_log2, to_cap;          // cap log2(e), scale / cap; 0: not capped
    // the chunk kernel's polynomials: s (near_c[0] + near_c[1] s^2 + near_c[2] s^4) for |s| below near, s P((s to_cap)^2)
    // below far
    float near, near_c[3], far, far_c[5];
    const float* slopes;             // device, [n][q_heads], or nullptr
};

inline ScoreArgs score_args(const AttnCall& c, bool precise)
{
    ScoreArgs a{};
    if (!c.scores) return a;
    a.slopes = c.scores->slopes;
    const double cap = c.scores->cap;
    if (cap > 0) {
        const double z = c.scale / cap;   // tanh's argument, for a score of 1
        a.cap_log2 = c.scores->cap * kLog2e;
        a.to_cap = (float)z;
        // tanh(z) / z = 1 - t / 3 + 2 t^2 / 15 - 17 t^3 / 315 + 62 t^4 / 2835, t = z^2.  For z below r the third power is
        // replaced by what the Chebyshev polynomial T3, put so that it is 0 at t = 0 and 1 at t = r^2, leaves of it, (the
        // fourth by t times that): off by 17 / 1260 (r^2 / (1 + w))^3 of tanh, w = sqrt(3) / 2 (checked up to r = 0.45).
        // r: as far as that is less than 2^-13 in base 2, with two parts 2^-20
        const double w = sqrt(3.0) / 2, limit = precise ? 0x1p-20 : 0x1p-13;
        const double r = fmin(0.45, pow(limit * 1260 / 17 * pow(1 + w, 3) / (cap * kLog2e), 1.0 / 7)), b = (1 + w) / (r * r);
        const double near[3] = {1.0, -1.0 / 3 + 17.0 / 315 * 1.5 / (b * b) - 62.0 / 2835 * 4.5 * w / (b * b * b),
                                2.0 / 15 - 17.0 / 315 * 3 * w / b + 62.0 / 2835 * 5.25 / (b * b)};
        const double far[5] = {1.0, -0.33329667636182275, 0.13268236858747265, -0.05027794750116984, 0.013105829772149474};
        const double unit = c.scale * kLog2e;
        // powers stay finite; |y| stays below kBound
        a.near = (float)fmin(fmin(r / z, (a.slopes ? kBiasedBound : kBound) / unit), 1e9);
        for (int i = 0; i < 3; ++i) a.near_c[i] = (float)(unit * pow(z, 2 * i) * near[i]);
        if (!std::isfinite(a.near_c[2])) a.near = 0.0f;   // no score is below it
        a.far = (float)(0.75 / z);
        for (int i = 0; i < 5; ++i) a.far_c[i] = (float)(unit * far[i]);
    }
    return a;
}

template <typename B>
B batch_args_as(const KvCache& kv, const ar_batch_t& b, const AttnCall& c)
{
    B x;
    static_cast<BatchArgs&>(x) = batch_args(kv, b, c.window);
    if constexpr (std::is_same<B, MaskedBatchArgs>::value) {
        x.prefix = c.scores->prefix;
        x.first = c.scores->first;
    }
    return x;
}

// 16-byte chunk `c` of 128-byte row `r` of a panel written by a tensor copy
// with the 128-byte swizzle (the panel starts on a multiple of 1024 bytes).
__device__ __forceinline__ uint32_t swizzled(uint32_t panel, int r, int c)
{
    return panel + r * 128 + ((c ^ (r & 7)) << 4);
}

}  // namespace argb
