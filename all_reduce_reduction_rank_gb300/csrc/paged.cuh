// Device helpers of the paged-cache kernels: a sequence's place in the batch,
// the split of a call's key tiles over the CTAs, tensor copies of pages, and
// bounded waits.
#pragma once

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

__device__ __forceinline__ Seq load_seq(const BatchArgs& b, int s, DevStatus* st) { return check_seq(b, read_seq(b, s), st); }

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
template <typename S>
__device__ __forceinline__ void enter_sequence(const BatchArgs& b, int tm, const Seq& q, u64 g, u64 off, Cursor& c)
{
    const int lane = threadIdx.x & 31;
    auto units_of = [&](int t) { return (unsigned)(span_of<S::KT>(q, tm, t, b.window).tiles + S::W); };
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
template <typename S>
__device__ bool split_few(const BatchArgs& b, int tm, int heads, int min_units, Cursor& c, Seq& at, DevStatus* st)
{
    const int lane = threadIdx.x & 31;
    const int per = (b.seqs + 31) / 32, s0 = min(lane * per, b.seqs), s1 = min(s0 + per, b.seqs);
    auto units_in = [&](const Seq& q) { return units_of_sequence<S>(q, tm, b.window); };
    u64 mine = 0;
    Seq q{0, 0, 0, 0};
    if (per == 1) {
        if (s0 < s1) {
            q = load_seq(b, s0, st);
            mine = units_in(q);
        }
    } else {
        RawSeq raw[8];   // all loads before the first use: a report orders what follows it
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (s0 + k < s1) raw[k] = read_seq(b, s0 + k);
#pragma unroll 1
        for (int k = 0; k < per; ++k) {
            if (s0 + k < s1) mine += units_in(check_seq(b, raw[0], st));
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
            const u64 u = units_in(q);
            if (off < u) break;
            off -= u;
        }
    c.s = __shfl_sync(0xffffffffu, s, src);
    off = __shfl_sync(0xffffffffu, off, src);
    at.q0 = __shfl_sync(0xffffffffu, q.q0, src);
    at.nq = __shfl_sync(0xffffffffu, q.nq, src);
    at.len = __shfl_sync(0xffffffffu, q.len, src);
    at.c0 = __shfl_sync(0xffffffffu, q.c0, src);
    enter_sequence<S>(b, tm, at, g, off, c);
    return true;
}

// Called by all NT threads; false for a CTA with nothing to do.  `min_units`:
// a run is at least that long, so that small calls do not pay for joins.  `at`:
// the sequence the run begins in.
template <typename S, int NT>
__device__ bool split_work(const BatchArgs& b, int tm, int heads, int min_units, SplitShared* sh, Cursor& c, Seq& at,
                           DevStatus* st)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    // consecutive sequences for a warp's lanes; few sequences are spread over the warps
    const int of_warp = (b.seqs + NT / 32 - 1) / (NT / 32), per = (of_warp + 31) / 32;
    const int w0 = min(warp * of_warp, b.seqs), w1 = min(w0 + of_warp, b.seqs);
    const int s0 = min(w0 + lane * per, w1), s1 = min(s0 + per, w1);
    auto units_of = [&](const Seq& q, int t) { return (unsigned)(span_of<S::KT>(q, tm, t, b.window).tiles + S::W); };
    u64 mine = 0;
    // long sequences' row tiles are counted by the whole warp
    for (int k = 0; k < per; ++k) {
        const int s = s0 + k;
        Seq q{0, 0, 0, 0};
        if (s < s1) q = load_seq(b, s, st);
        const int nt = (q.nq + tm - 1) / tm;
        const bool is_long = nt > 8;
        if (!is_long) mine += units_of_sequence<S>(q, tm, b.window);
        unsigned todo = __ballot_sync(0xffffffffu, is_long);
        while (todo) {
            const int src = __ffs(todo) - 1;
            todo &= todo - 1;
            Seq w;
            w.q0 = 0;
            w.nq = __shfl_sync(0xffffffffu, q.nq, src);
            w.len = __shfl_sync(0xffffffffu, q.len, src);
            w.c0 = w.len - w.nq;
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
            if (s + 1 < s1) sum = units_of_sequence<S>(load_seq(b, s, st), tm, b.window);
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
struct Segment {
    Seq q;
    Span span;
    int head, s, t;
    int j0, j1;                       // key tiles of this CTA
    unsigned first_cta, parts, slot;  // CTA of its first part, its parts (1: whole), this CTA's partial slot
};

// Walks a run.  Every warp keeps its own copy; all read the same values.
template <typename S>
struct Walk {
    Cursor c;
    Seq q;
    int loaded;

    Walk() = default;   // in shared memory
    __device__ __forceinline__ Walk(const Cursor& cur, const Seq& at) : c(cur), q(at), loaded(cur.s) {}

    __device__ __forceinline__ bool next(const BatchArgs& b, int tm, Segment& seg, DevStatus* st)
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
            seg.span = span_of<S::KT>(q, tm, c.t, b.window);
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

// 16-byte chunk `c` of 128-byte row `r` of a panel written by a tensor copy
// with the 128-byte swizzle (the panel starts on a multiple of 1024 bytes).
__device__ __forceinline__ uint32_t swizzled(uint32_t panel, int r, int c)
{
    return panel + r * 128 + ((c ^ (r & 7)) << 4);
}

}  // namespace argb
