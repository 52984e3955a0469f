// A step's batch made on the device: token ranges, lengths, page tables and
// slots from the requests' lengths and a stack of free pages.
//
// Three running sums over the sequences (new tokens, pages taken, pages given
// back) place everything: page i that is taken is entry top - 1 - i of the stack,
// page i that comes back goes to entry count + i.  Integers only; a few KB move,
// so what bounds it is the chain launch -> lengths -> sums -> stack -> table.
//
// One CTA does all of it for up to 1024 sequences, a thread a sequence: the
// sums take one barrier, and nothing is written before the totals are known, so
// that a step that cannot be served changes nothing.  Where a sequence moves several
// pages, or has several new tokens, threads share the pages (tokens) of all sequences
// and look up whose each is; for many tokens (kWide) the threads of a cluster's CTAs,
// each of which takes the sums for itself.  More sequences go through one CTA in
// chunks, once for the totals, once for the pages given back, once for the rest, and
// their rows, or those of very many tokens (kRowsHere), take a second launch.
// Measured on GB300: one sequence 2.0 us, 300 slots of which 27 are over and 6 take prompts (3852 tokens) 6.7, 60000
// tokens of 7 prompts with 1900 pages given back 8.5.
#include <algorithm>

#include "cluster.cuh"
#include "kv_step.cuh"
#include "paged.cuh"

namespace argb {
namespace {

constexpr int kTh = 1024;
constexpr int kRowTh = 256;
// Measured on GB300, us in one CTA / a cluster of 8 / by a second launch: 4 sequences of 64 tokens 3.0 / 3.7 / 4.0, of
// 256 3.9 / 4.7 / 4.6, of 512 4.5 / 4.7 / 4.6, of 1000 6.0 / 4.7 / 4.6, of 4000 15 / 5.8 / 5.0; 60000 tokens with as many
// pages given back 49 / 12 / 8.4.  1000 sequences of one token 3.0 in one CTA, one 1.9.  (A second launch costs the host
// as much again: it is for where the rows are many.)
constexpr unsigned kClusterCtas = 8;
constexpr size_t kWide = 2048;       // tokens from which a cluster shares the work
constexpr size_t kRowsHere = 16384;  // tokens whose rows the first launch writes
constexpr uint32_t kMost = 0x7fffffffu;   // sums stop here: beyond every limit they are held against

struct StepArgs {
    const int32_t* new_len;
    const int32_t* done;
    const int32_t* kv_len;
    int32_t* kv_len_out;
    int32_t* table;
    size_t table_stride;
    int32_t* free_pages;
    const int32_t* free_count;
    int32_t* free_count_out;
    int32_t* q_start;
    long long* slots;
    int32_t* positions;
    int seqs, tokens, capacity;
    int longest;                 // tokens that a table row can hold
    int page_shift, pages;
    bool rows_here;
};

__device__ __forceinline__ uint32_t add_most(uint32_t a, uint32_t b) { return min(a + b, kMost); }

__device__ __forceinline__ Sums add(const Sums& a, const Sums& b)
{
    return Sums{add_most(a.tokens, b.tokens), add_most(a.take, b.take), add_most(a.give, b.give), a.flags | b.flags};
}

__device__ __forceinline__ One read_one(const StepArgs& a, int s)
{
    if (s >= a.seqs) return One{0, 0, 0, Sums{0, 0, 0, 0}};
    return one_of(a.kv_len[s], a.new_len[s], a.done && a.done[s] != 0, a.longest, a.page_shift);
}

struct StepShared {
    Sums warp[32];
    uint32_t end[kTh];           // inclusive sums of the pages or tokens being shared out
    int kept[kTh];
};

__device__ __forceinline__ Sums shfl_up(const Sums& x, int by)
{
    return Sums{__shfl_up_sync(0xffffffffu, x.tokens, by), __shfl_up_sync(0xffffffffu, x.take, by),
                __shfl_up_sync(0xffffffffu, x.give, by), 0u};
}

// Inclusive sums over the CTA's threads; `total`: of all of them, with all flags.
// (A barrier lies between two calls' uses of the shared words.)
__device__ __forceinline__ Sums scan(const Sums& x, StepShared* sh, Sums& total)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    auto up = [&](Sums v) {
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const Sums y = shfl_up(v, o);
            if (lane >= o) v = add(v, y);
        }
        return v;
    };
    Sums in = up(x);
    const uint32_t flags = __reduce_or_sync(0xffffffffu, x.flags);
    if (lane == 31) {
        sh->warp[warp] = in;
        sh->warp[warp].flags = flags;
    }
    __syncthreads();
    const Sums w = lane < warps ? sh->warp[lane] : Sums{0, 0, 0, 0};
    const Sums all = up(w);
    auto of = [&](int from) {
        return Sums{__shfl_sync(0xffffffffu, all.tokens, from), __shfl_sync(0xffffffffu, all.take, from),
                    __shfl_sync(0xffffffffu, all.give, from), 0u};
    };
    total = of(31);
    total.flags = __reduce_or_sync(0xffffffffu, w.flags);
    const Sums before = of((warp + 31) & 31);
    if (warp > 0) in = add(in, before);
    return in;
}

// The thread whose share of the sums holds item i: the first with end > i.
__device__ __forceinline__ int owner(const uint32_t* end, int n, uint32_t i)
{
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (end[mid] > i)
            hi = mid;
        else
            lo = mid + 1;
    }
    return lo;
}

// f(i) for the thread's items i of [0, n), shared by all CTAs, then store(i, what f gave): four loads in flight at once.
template <typename F, typename S>
__device__ __forceinline__ void share_out(uint32_t n, F&& f, S&& store)
{
    const uint32_t step = gridDim.x * blockDim.x;
    for (uint32_t i0 = blockIdx.x * blockDim.x + threadIdx.x; i0 < n; i0 += 4 * step) {
        decltype(f(0u)) v[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (i0 + k * step < n) v[k] = f(i0 + k * step);
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (i0 + k * step < n) store(i0 + k * step, v[k]);
    }
}

__device__ __forceinline__ void write_row(const StepArgs& a, int t, long long slot, int position)
{
    if (a.slots) a.slots[t] = slot;
    if (a.positions) a.positions[t] = position;
}

// The slot of `position` in page `page`; -1 for a page that is not in the caches.
__device__ __forceinline__ long long slot_of(const StepArgs& a, int page, int position, DevStatus* st)
{
    if (page < 0 || page >= a.pages) {
        report_index(st);
        return -1;
    }
    return ((long long)page << a.page_shift) + (position & ((1 << a.page_shift) - 1));
}

// Every CTA has come here, and sees what the others wrote before.
__device__ __forceinline__ void sync_all()
{
    if (gridDim.x > 1) {
        cluster_arrive();
        cluster_wait();
    } else {
        __syncthreads();
    }
}

// One CTA, or one cluster of them for up to a CTA's threads of sequences.
__global__ void __launch_bounds__(kTh)
kv_step_kernel(const __grid_constant__ StepArgs a, DevStatus* st)
{
    __shared__ StepShared sh;
    const int tid = threadIdx.x, nt = blockDim.x;
    pdl_acquire();
    pdl_release();   // few CTAs: the next launch's may wait beside them
    const bool lead = blockIdx.x == 0;
    const uint32_t me = blockIdx.x * nt + tid, everyone = gridDim.x * nt;
    const int count = *a.free_count;
    const int chunks = (a.seqs + nt - 1) / nt;
    One o = read_one(a, tid);
    // a single new token in a page that the sequence has (-1: it does not, or its lengths are
    // refused): on its way while the sums are taken
    const int entry = entry_of_one(o, a.page_shift);
    int page = -1;
    if (a.rows_here && entry >= 0) page = a.table[(size_t)tid * a.table_stride + entry];
    Sums in, total;
    if (chunks <= 1) {
        in = scan(o.x, &sh, total);
    } else {
        Sums mine = o.x;
        for (int c = 1; c < chunks; ++c) mine = add(mine, read_one(a, c * nt + tid).x);
        scan(mine, &sh, total);
    }
    const bool bad = (total.flags & kBad) || count < 0 || count > a.capacity || total.tokens > (uint32_t)a.tokens ||
                     total.give > (uint32_t)(a.capacity - count);
    const bool empty = bad || total.take > (uint32_t)count + total.give;
    if (empty) {
        if (me == 0) {
            if (bad)
                report_index(st);
            else
                atomicCAS(&st->code, 0, AR_ERR_PAGES);
            *a.free_count_out = count;
            a.q_start[a.seqs] = 0;
        }
        for (int s = tid; lead && s < a.seqs; s += nt) {
            a.q_start[s] = 0;
            a.kv_len_out[s] = a.kv_len[s];   // (in place: no change)
        }
        if (a.rows_here)
            for (uint32_t t = me; t < (uint32_t)a.tokens; t += everyone) write_row(a, (int)t, -1, -1);
        return;
    }
    if (gridDim.x > 1) sync_all();   // all have read the lengths, which may be written in place

    // the pages of the sequences that are over, onto the stack
    if (total.give > 0) {
        uint32_t before = 0;
        for (int c = 0; c < chunks; ++c) {
            Sums here = total;
            if (chunks > 1) {
                o = read_one(a, c * nt + tid);
                __syncthreads();
                in = scan(o.x, &sh, here);
            }
            sh.end[tid] = in.give;
            __syncthreads();
            share_out(
                here.give,
                [&](uint32_t i) {
                    const int w = owner(sh.end, nt, i);
                    const uint32_t j = i - (w > 0 ? sh.end[w - 1] : 0u);
                    return a.table[(size_t)(c * nt + w) * a.table_stride + j];
                },
                [&](uint32_t i, int page) { a.free_pages[(uint32_t)count + before + i] = page; });
            before += here.give;
            sync_all();
        }
    }

    // pages off its top, lengths and ranges
    const uint32_t top = (uint32_t)count + total.give;
    uint32_t taken = 0, first = 0;
    for (int c = 0; c < chunks; ++c) {
        Sums here = total;
        if (chunks > 1) {
            o = read_one(a, c * nt + tid);
            __syncthreads();
            in = scan(o.x, &sh, here);
        }
        const int s = c * nt + tid;
        int32_t* row = a.table + (size_t)s * a.table_stride;
        if (!(here.flags & kSeveralPages)) {
            if (lead && o.x.take == 1) {
                page = a.free_pages[top - (taken + in.take)];
                row[(o.kept + (1 << a.page_shift) - 1) >> a.page_shift] = page;
            }
        } else {
            sh.end[tid] = in.take;
            sh.kept[tid] = (int)((uint32_t)(o.kept + (1 << a.page_shift) - 1) >> a.page_shift);
            __syncthreads();
            struct Entry {
                int32_t* at;
                int page;
            };
            share_out(
                here.take,
                [&](uint32_t i) {
                    const int page = a.free_pages[top - 1 - (taken + i)];
                    const int w = owner(sh.end, nt, i);
                    const uint32_t j = i - (w > 0 ? sh.end[w - 1] : 0u);
                    return Entry{a.table + (size_t)(c * nt + w) * a.table_stride + sh.kept[w] + j, page};
                },
                [&](uint32_t, const Entry& x) { *x.at = x.page; });
        }
        if (lead && s < a.seqs) {
            a.q_start[s] = (int)(first + in.tokens - o.x.tokens);
            a.kv_len_out[s] = o.kept + o.added;
        }
        taken += here.take;
        first += here.tokens;
        if (a.rows_here && !(total.flags & kSeveralTokens)) {
            if (lead && o.added == 1) write_row(a, (int)in.tokens - 1, slot_of(a, page, o.kept, st), o.kept);
        } else if (a.rows_here) {                           // of one chunk
            sync_all();                                     // the table's new entries; sh is free
            sh.end[tid] = in.tokens;
            sh.kept[tid] = o.kept;
            __syncthreads();
            struct Row {
                int place, page;
            };
            share_out(
                total.tokens,
                [&](uint32_t t) {
                    const int w = owner(sh.end, nt, t);
                    const int p = sh.kept[w] + (int)(t - (w > 0 ? sh.end[w - 1] : 0u));
                    return Row{p, a.table[(size_t)w * a.table_stride + (p >> a.page_shift)]};
                },
                [&](uint32_t t, const Row& x) { write_row(a, (int)t, slot_of(a, x.page, x.place, st), x.place); });
        }
    }
    if (me == 0) {
        a.q_start[a.seqs] = (int)total.tokens;
        *a.free_count_out = (int)(top - total.take);
    }
    if (a.rows_here)
        for (uint32_t t = total.tokens + me; t < (uint32_t)a.tokens; t += everyone) write_row(a, (int)t, -1, -1);
}

// The rows of a step of many tokens, a thread a token.
__global__ void __launch_bounds__(kRowTh)
kv_rows_kernel(const __grid_constant__ StepArgs a, DevStatus* st)
{
    pdl_acquire();
    const int lane = threadIdx.x & 31;
    const int t = blockIdx.x * kRowTh + threadIdx.x, w0 = t - lane;
    const int total = a.q_start[a.seqs];
    if (w0 < total) {
        // the sequences of the warp's tokens, then each lane's among them
        int lo = seq_of(a.q_start, a.seqs, w0, lane), hi = lo;
        if (a.q_start[lo + 1] <= min(w0 + 31, total - 1)) hi = seq_of(a.q_start, a.seqs, min(w0 + 31, total - 1), lane);
        if (t < total) {
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (a.q_start[mid] <= t)
                    lo = mid;
                else
                    hi = mid - 1;
            }
            const int p = a.kv_len_out[lo] - (a.q_start[lo + 1] - t);
            const int page = a.table[(size_t)lo * a.table_stride + (p >> a.page_shift)];
            write_row(a, t, slot_of(a, page, p, st), p);
        }
    }
    if (t >= total && t < a.tokens) write_row(a, t, -1, -1);
}

}  // namespace

int launch_kv_step(KvCache& kv, const ar_kv_step_t& x, uint64_t moved, int* launches, cudaStream_t s)
{
    Handle& h = *kv.h;
    StepArgs a{};
    a.new_len = x.new_len;
    a.done = x.done;
    a.kv_len = x.kv_len;
    a.kv_len_out = x.kv_len_out;
    a.table = x.page_table;
    a.table_stride = x.table_stride;
    a.free_pages = x.free_pages;
    a.free_count = x.free_count;
    a.free_count_out = x.free_count_out;
    a.q_start = x.q_start;
    a.slots = reinterpret_cast<long long*>(x.slots);
    a.positions = x.positions;
    a.seqs = x.seqs;
    a.tokens = (int)x.tokens;
    a.capacity = (int)x.capacity;
    a.page_shift = page_shift(kv);
    a.longest = longest_row(x.table_stride, a.page_shift);
    a.pages = (int)kv.d.pages;
    const bool rows = x.tokens > 0 && (x.slots || x.positions);
    a.rows_here = rows && x.seqs <= kTh && x.tokens <= kRowsHere;
    const size_t want = std::max((size_t)x.seqs, x.tokens);
    const unsigned block = want >= (size_t)kTh ? kTh : (unsigned)((want + 127) / 128 * 128);
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = h.pdl ? 1 : 0;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = a.rows_here && x.tokens >= kWide ? kClusterCtas : 1;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(attr[1].val.clusterDim.x);
    cfg.blockDim = dim3(block ? block : 128);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    rec_begin(h, s);
    cudaError_t e = cudaLaunchKernelEx(&cfg, kv_step_kernel, a, h.status);
    *launches = 1;
    if (e == cudaSuccess && rows && !a.rows_here) {
        e = launch_kernel(h, kv_rows_kernel, dim3((unsigned)((x.tokens + kRowTh - 1) / kRowTh)), dim3(kRowTh), 0, s, a,
                          h.status);
        *launches = 2;
    }
    rec_end(h, s, AR_K_KV_STEP, moved, *launches);
    return e == cudaSuccess ? launch_status() : AR_ERR_CUDA;
}

}  // namespace argb
