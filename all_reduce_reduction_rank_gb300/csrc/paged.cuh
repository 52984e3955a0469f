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

// Values out of range reach no memory: a bad token range counts as no tokens,
// a bad length as no keys.
__device__ __forceinline__ Seq load_seq(const BatchArgs& b, int s, DevStatus* st)
{
    const int q0 = b.q_start[s], q1 = b.q_start[s + 1], len = b.kv_len[s];
    Seq r{q0, q1 - q0, len, 0};
    if (q0 < 0 || q1 < q0 || q1 > b.tokens) {
        report_index(st);
        r.q0 = r.nq = 0;
    }
    if (len < 0 || len > (1 << 30) || (size_t)len > (b.table_stride << b.page_shift)) {
        report_index(st);
        r.len = 0;
    }
    r.c0 = r.len - r.nq;
    return r;
}

// ---- split of the work ------------------------------------------------------------
// The unit is one tile of KT keys against one row tile: TM consecutive new
// tokens of a sequence, with the query heads of one head group.  A (sequence,
// row tile) pair counts its tiles between the first key any of its rows sees
// and the last; at least one, so that rows that see nothing are written too.
// The units of all (head group, sequence, row tile) triples, in that order,
// are cut into equal runs, one per CTA, whatever the lengths are: every CTA
// gets the same number of key tiles, and only the first and the last triple
// of its run can be shared with other CTAs.

struct Span {
    int key_lo, key_hi;   // keys that some row of the tile sees (key_hi <= key_lo: none)
    int j_lo, units;      // first key tile, number of tiles (>= 1)
};

template <int KT>
__device__ __forceinline__ Span span_of(const Seq& q, int tm, int t, int window)
{
    const int first = q.c0 + t * tm;                                // position of the tile's first token
    const int last = q.c0 + min((t + 1) * tm, q.nq);                // one past its last token's position
    Span p;
    p.key_hi = max(last, 0);
    p.key_lo = window > 0 ? max(first - window + 1, 0) : 0;
    p.j_lo = p.key_lo / KT;
    p.units = max((p.key_hi + KT - 1) / KT - p.j_lo, 1);
    return p;
}

struct Cursor {
    unsigned long long g, end;   // next unit and one past the last of this CTA's run
    unsigned long long per_head; // units of one head group
    unsigned long long total;    // units of the call
    unsigned ctas;               // CTAs that share them
    int head, s, t, off;         // the triple that unit g is in, and its place in it
};

__device__ __forceinline__ unsigned long long run_begin(unsigned long long total, unsigned ctas, unsigned c)
{
    return total * c / ctas;
}

// The CTA whose run holds unit u.
__device__ __forceinline__ unsigned cta_of(unsigned long long total, unsigned ctas, unsigned long long u)
{
    return (unsigned)(((u + 1) * ctas - 1) / total);
}

struct SplitShared {
    unsigned long long warp_sum[32];
    unsigned long long total;
    unsigned long long off;
    int s;
};

// Called by all NT threads.  `min_units`: a run is at least that long (the
// last ones may be empty), so that small calls do not pay for joins.
template <int KT, int NT>
__device__ Cursor split_work(const BatchArgs& b, int tm, int heads, int min_units, SplitShared* sh, DevStatus* st)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (b.seqs + NT - 1) / NT;
    const int s0 = min(tid * per, b.seqs), s1 = min(s0 + per, b.seqs);
    unsigned long long mine = 0;
    // long sequences' row tiles are counted by the whole warp
    for (int k = 0; k < per; ++k) {
        const int s = s0 + k;
        Seq q{0, 0, 0, 0};
        if (s < s1) q = load_seq(b, s, st);
        const int nt = (q.nq + tm - 1) / tm;
        const bool is_long = nt > 8;
        if (!is_long)
            for (int t = 0; t < nt; ++t) mine += (unsigned)span_of<KT>(q, tm, t, b.window).units;
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
            unsigned long long sum = 0;
            for (int t = lane; t < wt; t += 32) sum += (unsigned)span_of<KT>(w, tm, t, b.window).units;
            for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            if (lane == src) mine += sum;
        }
    }
    unsigned long long incl = mine;
    for (int o = 1; o < 32; o <<= 1) {
        const unsigned long long x = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += x;
    }
    if (lane == 31) sh->warp_sum[warp] = incl;
    __syncthreads();
    unsigned long long before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < NT / 32; ++w) {
        if (w < warp) before += sh->warp_sum[w];
        all += sh->warp_sum[w];
    }
    Cursor c;
    c.per_head = all;
    c.total = all * (unsigned)heads;
    c.ctas = gridDim.x;
    const unsigned long long most = (c.total + min_units - 1) / min_units;
    if (most < c.ctas) c.ctas = (unsigned)most;
    c.g = c.end = 0;
    c.head = c.s = c.t = c.off = 0;
    if (blockIdx.x >= c.ctas) return c;   // the whole CTA
    c.g = run_begin(c.total, c.ctas, blockIdx.x);
    c.end = run_begin(c.total, c.ctas, blockIdx.x + 1);
    c.head = (int)(c.g / c.per_head);
    const unsigned long long in_head = c.g - c.head * c.per_head;
    const unsigned long long excl = before + incl - mine;
    if (in_head >= excl && in_head < excl + mine) {
        // this thread's sequences hold it
        unsigned long long at = excl;
        for (int s = s0; s < s1; ++s) {
            const Seq q = load_seq(b, s, st);
            const int nt = (q.nq + tm - 1) / tm;
            unsigned long long sum = 0;
            if (s + 1 < s1)
                for (int t = 0; t < nt; ++t) sum += (unsigned)span_of<KT>(q, tm, t, b.window).units;
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
    // the row tile inside the sequence: every warp walks it, 32 tiles at a time
    unsigned long long off = sh->off;
    const Seq q = load_seq(b, c.s, st);
    const int nt = (q.nq + tm - 1) / tm;
    for (int t0 = 0; t0 < nt; t0 += 32) {
        const int t = t0 + lane;
        unsigned long long u = t < nt ? (unsigned)span_of<KT>(q, tm, t, b.window).units : 0, in = u;
        for (int o = 1; o < 32; o <<= 1) {
            const unsigned long long x = __shfl_up_sync(0xffffffffu, in, o);
            if (lane >= o) in += x;
        }
        const unsigned here = __ballot_sync(0xffffffffu, in > off);
        if (here) {
            const int src = __ffs(here) - 1;
            c.t = t0 + src;
            c.off = (int)(off - __shfl_sync(0xffffffffu, in - u, src));
            break;
        }
        off -= __shfl_sync(0xffffffffu, in, 31);
    }
    return c;
}

// One triple's part in this CTA's run.
struct Segment {
    Seq q;
    Span span;
    int head, s, t;
    int j0, j1;                       // key tiles of this CTA
    bool whole;                       // the triple lies in this run entirely
    unsigned first_cta, parts, slot;  // if not whole: where it begins, its parts, this CTA's partial slot
};

// Walks a run.  Every warp keeps its own copy; all read the same values.
template <int KT>
struct Walk {
    Cursor c;
    Seq q;
    int loaded;

    Walk() = default;   // in shared memory
    __device__ __forceinline__ explicit Walk(const Cursor& cur) : c(cur), q{0, 0, 0, 0}, loaded(-1) {}

    __device__ __forceinline__ bool next(const BatchArgs& b, int tm, Segment& seg, DevStatus* st)
    {
        if (c.g >= c.end) return false;
        for (;;) {
            if (loaded != c.s) {
                q = load_seq(b, c.s, st);
                loaded = c.s;
            }
            if (c.t * tm < q.nq) break;
            c.t = 0;
            if (++c.s == b.seqs) {
                c.s = 0;
                ++c.head;
            }
        }
        seg.q = q;
        seg.span = span_of<KT>(q, tm, c.t, b.window);
        seg.head = c.head;
        seg.s = c.s;
        seg.t = c.t;
        const unsigned long long left = c.end - c.g;
        const int rest = seg.span.units - c.off;
        const int take = left < (unsigned long long)rest ? (int)left : rest;
        seg.j0 = seg.span.j_lo + c.off;
        seg.j1 = seg.j0 + take;
        seg.whole = take == seg.span.units;
        if (!seg.whole) {
            const unsigned long long begin = c.g - c.off;
            seg.first_cta = cta_of(c.total, c.ctas, begin);
            seg.parts = cta_of(c.total, c.ctas, begin + seg.span.units - 1) - seg.first_cta + 1;
            seg.slot = 2 * blockIdx.x + (seg.first_cta == blockIdx.x ? 1 : 0);
        }
        c.g += take;
        if (take == rest) {
            ++c.t;
            c.off = 0;
        } else {
            c.off += take;
        }
        return true;
    }
};

// Partial slot of part i of a triple that begins in CTA f.
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

__device__ __forceinline__ void mbar_arrive(uint64_t* bar)
{
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}

__device__ __forceinline__ void fence_proxy_async()
{
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// Bounded wait: false after about a second.
__device__ __forceinline__ bool wait_a_second(uint64_t* bar, uint32_t parity, volatile int* stop)
{
    // the clock is read after 256 polls only: reading it costs as much as a tile's products
    uint64_t t0 = 0;
    for (uint32_t i = 0; i < kMbarMaxPolls; ++i) {
        if (mbar_try_wait(bar, parity)) return true;
        if (stop && *stop) return false;
        if ((i & 255) == 255) {
            if (t0 == 0)
                t0 = globaltimer_ns();
            else if (globaltimer_ns() - t0 > 1000000000ull)
                return false;
        }
    }
    return false;
}

// The same for the warps of a CTA that depend on one another: it also ends
// once another warp has given up, and giving up sets the status word.
__device__ __forceinline__ bool wait_or_give_up(uint64_t* bar, uint32_t parity, volatile int* gave_up, DevStatus* st)
{
    if (wait_a_second(bar, parity, gave_up)) return true;
    *gave_up = 1;
    report_wait_timeout(st);
    return false;
}

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// 16-byte chunk `c` of 128-byte row `r` of a panel written by a tensor copy
// with the 128-byte swizzle (the panel starts on a multiple of 1024 bytes).
__device__ __forceinline__ uint32_t swizzled(uint32_t panel, int r, int c)
{
    return panel + r * 128 + ((c ^ (r & 7)) << 4);
}

}  // namespace argb
