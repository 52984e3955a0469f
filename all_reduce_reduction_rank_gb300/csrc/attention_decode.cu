// Paged attention for few query rows per kv head: decode steps of one token
// a sequence, or of a few drafted ones.
//
// A row tile holds at most 8 or 16 rows (new tokens x the query heads that share
// a kv head), and every key and value of the sequence is read for it once, so
// the bound is HBM: 4 D bytes per key and head against 64 D flops on a tile of 16,
// 16 flops per byte where the machine's tensor cores could do 280.  The
// products therefore use mma.sync m16n8k16, whose tiles waste least: S = Q K^T
// with 16 rows, and with 8 the transposed products S^T = K Q^T, O^T = V^T P^T,
// half as many (8 sequences of 700 keys, 8 heads a kv head: 12.2 us with 16 rows,
// 10.6 with 8).  The design is about keeping enough copies in flight: one warp issues tensor
// copies of 64-key tiles (K and V) into a ring of stages, two CTAs of an SM
// together holding about 190 KB of them, and four warps each take 16 keys of
// every tile with their own running maximum, sum and output accumulators, so
// nothing but the ring's barriers is shared until a row tile's keys end.
//
// Measured on GB300 (n = 8 bf16, heads of 128, 8 query heads a kv head): 64
// sequences of 1 to 8192 keys, 792 MB: 127 us, 6.25 TB/s (93% of the copy rate); 4
// sequences of 70 to 131 thousand keys (n = 4 fp16, 1.77 GB): 258 us, 6.86 TB/s
// (103%); one sequence of 1500 keys: 8.6 to 9.2 us, where launch, split, page, copy, two
// tiles and the join follow one another.  Short sequences are bound by the same
// chain per row tile (64 sequences of 300 keys: 25 us for 12.5 us of bytes); the
// tensor pipe is 14% busy at long ones, the warps wait for one another's results.
//
// Softmax in one pass, base 2: with x = scale log2(e) (q . k), a running
// reference m, p = 2^(x - m), l = sum p, o = sum p v.  m moves only when a row's
// maximum passes it by far (kSlack, kBelow), so the accumulators are seldom rescaled.
//
// Split of the keys: split_work cuts all key tiles of the call into equal runs,
// one per CTA.  Row tiles that lie in several runs leave their parts (o, m, l,
// fp32) in the workspace, and the CTA that arrives last joins them in the order
// of the keys, so the result does not depend on which one that is.
#include "paged.cuh"

namespace argb {
namespace {

constexpr int kKeys = 64;                    // keys of a tile
constexpr int kWarps = 4;                    // consumers, 16 keys each
constexpr int kTh = 32 * (kWarps + 1);

// a row tile's start and end weigh a key tile more (0 / 1 / 2 / 3: 8 sequences of 700
// keys 15.1 / 12.6 / 13.4 / 14.1 us, 64 of 1000 keys 59 / 55.5 / 53.5 / 53.0)
using DecodeSplit = Split<kKeys, 1, 4>;

template <int D> constexpr int kTileBytes = kKeys * D * 2;
// per SM.  With 8 rows three CTAs of two stages fit as well: 16.5 for 13.9 us at one sequence of
// 8000 keys (n = 2, 4 kv heads), 27.0 for 25.1 at 64 of 300, 124.5 for 127 at 64 of 1 to 8192.
constexpr int kCtas = 2;
template <int D> constexpr int kStages = 3 * (128 / D);
template <int ROWS, int D> constexpr int kAccStride = ROWS == 8 ? D + 4 : D;   // floats; + 4: no bank conflicts
template <int ROWS, int D> constexpr int kPartFloats = ROWS * (D + 2);

struct DecodeShared {
    uint64_t full[6], empty[6];
    float m[kWarps][16], l[kWarps][16];
    float top[16], sum[16];
    SplitShared split;
    int gave_up, last;
};
static_assert(sizeof(DecodeShared) <= 1024, "the shared memory of an SM's CTAs fits it exactly");

// stages, then two accumulator buffers, then DecodeShared
template <int ROWS, int D>
constexpr int kSmem = kStages<D> * 2 * kTileBytes<D> + 2 * ROWS * kAccStride<ROWS, D> * 4 + 1024;

struct DecodeArgs {
    const void* q[kMaxRanks];
    void* out[kMaxRanks];
    const CUtensorMap* maps;
    float* partial;
    unsigned* arrived;
    size_t q_stride, out_stride;
    float scale_log2;
    int n, kv_heads, group;                  // query heads per kv head
    int tile_heads, head_groups, tm;         // query heads and new tokens of a row tile
    int box_tokens, min_units;
    bool few;                                // split_few
};

template <int DT>
__device__ __forceinline__ void mma16816(float* d, const uint32_t* a, uint32_t b0, uint32_t b1)
{
    if constexpr (DT == AR_BF16)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                     "{%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                     "{%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void ldmatrix4(uint32_t* r, uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

__device__ __forceinline__ void ldmatrix4_trans(uint32_t* r, uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

// Transposes an 8 x 8 matrix of 16-bit elements, two of a row a thread.
__device__ __forceinline__ uint32_t transpose8(uint32_t x)
{
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

__device__ __forceinline__ void consumers_sync() { asm volatile("bar.sync 1, %0;" ::"n"(32 * kWarps) : "memory"); }

// A segment's rows: rank, kv head, first query head and number of heads, first
// new token, number of rows (row i: token i / heads, head i % heads).
struct RowTile {
    int rank, kv_head, head0, heads, tok0, rows;
};

__device__ __forceinline__ RowTile row_tile(const DecodeArgs& a, const Segment& seg)
{
    RowTile r;
    const int hg = seg.head % a.head_groups, kvh = seg.head / a.head_groups;
    r.kv_head = kvh % a.kv_heads;
    r.rank = kvh / a.kv_heads;
    r.heads = min(a.tile_heads, a.group - hg * a.tile_heads);
    r.head0 = r.kv_head * a.group + hg * a.tile_heads;
    r.tok0 = seg.t * a.tm;
    r.rows = min(a.tm, seg.q.nq - r.tok0) * r.heads;
    return r;
}

template <int D>
__device__ void produce(const DecodeArgs& a, const BatchArgs& b, const Cursor& cur, const Seq& at, uint8_t* stages,
                        DecodeShared* sh, DevStatus* st)
{
    const int lane = threadIdx.x & 31;
    const int per_page = kKeys / a.box_tokens;         // boxes of a tile along the keys: 1, 2 or 4
    const int panels = D / 64;
    // lane -> one copy of the tile
    const int box = lane % per_page, panel = (lane / per_page) % panels, is_v = lane / (per_page * panels);
    const bool mine = is_v < 2;
    Walk<DecodeSplit> walk(cur, at);
    Segment seg;
    int stage = 0;
    uint32_t phase = 0;
    uint32_t issued = 0;
    bool ok = true;
    while (ok && walk.next(b, a.tm, seg, st)) {
        const RowTile rt = row_tile(a, seg);
        if (rt.rank == b.absent) break;
        const CUtensorMap* map = a.maps + (is_v ? a.n : 0) + rt.rank;
        const int32_t* row = b.table + (size_t)seg.s * b.table_stride;
        for (int j = seg.j0; ok && j < seg.j1; ++j) {
            const int key = j * kKeys + box * a.box_tokens;
            bool copy = mine && key < seg.span.key_hi && key + a.box_tokens > seg.span.key_lo;
            int page = 0;
            if (copy) {
                page = row[key >> b.page_shift];
                if (page < 0 || page >= b.pages) {
                    report_index(st);
                    copy = false;
                }
            }
            if (issued >= (uint32_t)kStages<D>) ok = wait_or_give_up(&sh->empty[stage], phase ^ 1, &sh->gave_up, st);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            const int copies = __popc(__ballot_sync(0xffffffffu, copy));
            if (lane == 0) mbar_arrive_expect_tx(&sh->full[stage], (uint32_t)copies * a.box_tokens * 128u);
            __syncwarp();
            if (copy)
                page_copy(stages + (size_t)stage * 2 * kTileBytes<D> + is_v * kTileBytes<D> + panel * (kKeys * 128) +
                              box * a.box_tokens * 128,
                          map, panel * 64, key & ((1 << b.page_shift) - 1), rt.kv_head, page, &sh->full[stage]);
            ++issued;
            if (++stage == kStages<D>) {
                stage = 0;
                phase ^= 1;
            }
        }
    }
    wait_for_ring(sh->full, kStages<D>, issued, stage, phase, st);
}

template <int DT, int D, int ROWS>
__device__ void consume(const DecodeArgs& a, const BatchArgs& b, const Cursor& cur, const Seq& at, uint8_t* stages, float* acc,
                        DecodeShared* sh, DevStatus* st)
{
    using T = typename Payload<DT>::scalar_t;
    constexpr int KS = D / 16;      // k-steps of q . k
    constexpr int NT = ROWS == 8 ? D / 16 : D / 8;   // tiles of the output: 16 of D by 8 rows, or 16 rows by 8 of D
    constexpr int AS = kAccStride<ROWS, D>;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int r0 = lane >> 2, col = (lane & 3) * 2;
    // the two rows whose statistics this thread keeps, and the lanes it shares them with
    auto row_of = [&](int i) { return ROWS == 8 ? col + i : r0 + 8 * i; };
    constexpr int SHARED = ROWS == 8 ? 3 : 2, FIRST = ROWS == 8 ? 4 : 1;   // log2 of the lanes, first lane bit
    Walk<DecodeSplit> walk(cur, at);
    Segment seg;
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;   // false once a wait ran out: the warps still meet at every barrier, without the work
    while (walk.next(b, a.tm, seg, st)) {
        const RowTile rt = row_tile(a, seg);
        const T* qp = static_cast<const T*>(a.q[rt.rank]) + (size_t)rt.head0 * D;
        int limit[2], lower[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int r = row_of(i);
            limit[i] = r < rt.rows ? seg.q.c0 + rt.tok0 + r / rt.heads + 1 : 0;
            lower[i] = b.window > 0 ? limit[i] - b.window : 0;
        }
        // q, the fragments of rows r0 (and r0 + 8)
        uint32_t qf[KS][ROWS / 4];
#pragma unroll
        for (int i = 0; i < ROWS / 8; ++i) {
            const int r = r0 + 8 * i;
            const bool there = r < rt.rows;
            const int tok = rt.tok0 + r / rt.heads, hd = r % rt.heads;
            const T* row = qp + (size_t)(seg.q.q0 + tok) * a.q_stride + (size_t)hd * D + col;
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                qf[k][i] = there ? *reinterpret_cast<const uint32_t*>(row + 16 * k) : 0u;
                qf[k][ROWS / 8 + i] = there ? *reinterpret_cast<const uint32_t*>(row + 16 * k + 8) : 0u;
            }
        }
        // keys that every row of the tile sees
        const int last_tok = rt.tok0 + (rt.rows - 1) / rt.heads;
        const int all_hi = seg.q.c0 + rt.tok0 + 1;
        const int all_lo = b.window > 0 ? seg.q.c0 + last_tok + 1 - b.window : 0;
        float o[NT][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
#pragma unroll
        for (int n = 0; n < NT; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.0f;

        for (int j = seg.j0; j < seg.j1; ++j) {
            const int key0 = j * kKeys + warp * 16;
            if (ok) ok = wait_or_give_up(&sh->full[stage], phase, &sh->gave_up, st);
            ok = __all_sync(0xffffffffu, ok);
            if (ok && key0 < seg.span.key_hi && key0 + 16 > seg.span.key_lo) {
                const uint32_t kbase = smem_addr(stages + (size_t)stage * 2 * kTileBytes<D>);
                const uint32_t vbase = kbase + kTileBytes<D>;
                if (key0 + 16 > seg.span.key_hi || key0 < seg.span.key_lo) {
                    // slots of these pages that no row sees may hold anything: their values count as 0
                    for (int i = lane; i < 16 * (D / 8); i += 32) {
                        const int r = i / (D / 8), c = i % (D / 8);
                        if (key0 + r >= seg.span.key_hi || key0 + r < seg.span.key_lo) {
                            const uint32_t at = swizzled(vbase + (c >> 3) * (kKeys * 128), warp * 16 + r, c & 7);
                            asm volatile("st.shared.v4.b32 [%0], {%1,%1,%1,%1};" ::"r"(at), "r"(0) : "memory");
                        }
                    }
                    __syncwarp();
                    fence_proxy_async();   // before the next copy into this stage
                }
                // scores of 16 keys: S^T (16 keys by 8 rows), or S (16 rows by two times 8 keys); element e
                // of s[nt] is row_of(ROW(e)) and key KEY(nt, e).  Two chains of products for each
                // (3% on short rows).
                constexpr int NS = ROWS / 8;
                auto row_i = [](int e) { return ROWS == 8 ? e & 1 : e >> 1; };
                auto key_of = [&](int nt, int e) { return ROWS == 8 ? r0 + 8 * (e >> 1) : 8 * nt + col + (e & 1); };
                float s[NS][4] = {}, odd[NS][4] = {};
                const int hi8 = (lane >> 4) << 3, mid8 = (lane >> 3) & 1;
                const int kr = warp * 16 + (lane & 7) + (ROWS == 8 ? mid8 * 8 : hi8);
                const int kc = ROWS == 8 ? lane >> 4 : mid8;                  // low, high 8 of the k-step
#pragma unroll
                for (int k = 0; k < KS; ++k) {
                    uint32_t kf[4];
                    const int c = 2 * k + kc;
                    ldmatrix4(kf, swizzled(kbase + (c >> 3) * (kKeys * 128), kr, c & 7));
                    if constexpr (ROWS == 8) {
                        mma16816<DT>(k & 1 ? odd[0] : s[0], kf, qf[k][0], qf[k][1]);
                    } else {
                        mma16816<DT>(k & 1 ? odd[0] : s[0], qf[k], kf[0], kf[1]);
                        mma16816<DT>(k & 1 ? odd[1] : s[1], qf[k], kf[2], kf[3]);
                    }
                }
                const bool masked = key0 + 16 > all_hi || key0 < all_lo;
                float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
                for (int nt = 0; nt < NS; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float x = (s[nt][e] + odd[nt][e]) * a.scale_log2;
                        const int i = row_i(e);
                        if (masked) {
                            const int key = key0 + key_of(nt, e);
                            if (key >= limit[i] || key < lower[i]) x = -INFINITY;
                        }
                        s[nt][e] = x;
                        mx[i] = fmaxf(mx[i], x);
                    }
                bool move = false;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
#pragma unroll
                    for (int w = 0; w < SHARED; ++w) mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], FIRST << w));
                    move |= mx[i] > m[i] + (kSlack + kBelow<DT>);
                }
                if (__any_sync(0xffffffffu, move)) {
                    float f[2];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float to = fmaxf(m[i], mx[i] - kBelow<DT>);
                        f[i] = m[i] == -INFINITY ? 0.0f : ex2(m[i] - to);
                        m[i] = to;
                        l[i] *= f[i];
                    }
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int e = 0; e < 4; ++e) o[n][e] *= f[row_i(e)];
                }
                float p[NS][4];
#pragma unroll
                for (int nt = 0; nt < NS; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int i = row_i(e);
                        const float ref = m[i] == -INFINITY ? 0.0f : m[i];
                        p[nt][e] = ex2(s[nt][e] - ref);
                        l[i] += p[nt][e];
                    }
                // The product's operand has the cache's type: p = high + low, both rounded to it, so that
                // what is lost is a half step of a half step (fp16: or 2^-32 of the largest p, see kBelow).
                // Rounded once, the outputs of short batches were off by 1.4 times their own rounding;
                // the second product is hidden behind the copies.
                uint32_t high[2 * NS], low[2 * NS];
#pragma unroll
                for (int nt = 0; nt < NS; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; e += 2) {
                        float back[2];
                        const uint32_t w = Payload<DT>::narrow(&p[nt][e]);
                        Payload<DT>::widen(w, back);
                        back[0] = p[nt][e] - back[0];
                        back[1] = p[nt][e + 1] - back[1];
                        high[2 * nt + e / 2] = w;
                        low[2 * nt + e / 2] = Payload<DT>::narrow(back);
                    }
                if constexpr (ROWS == 8) {
                    // O^T += V^T P^T: the scores' place holds P^T by rows, the operand wants it by columns
                    const uint32_t h0 = transpose8(high[0]), h1 = transpose8(high[1]);
                    const uint32_t l0 = transpose8(low[0]), l1 = transpose8(low[1]);
                    const int vr = warp * 16 + (lane & 7) + hi8;    // keys 0-7, 8-15
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        uint32_t vf[4];
                        const int c = 2 * n + mid8;                 // low, high 8 of the 16 columns
                        ldmatrix4_trans(vf, swizzled(vbase + (c >> 3) * (kKeys * 128), vr, c & 7));
                        mma16816<DT>(o[n], vf, h0, h1);
                        mma16816<DT>(o[n], vf, l0, l1);
                    }
                } else {
                    const int vr = warp * 16 + (lane & 15);         // keys 0-7, 8-15
                    const int vc = lane >> 4;                       // columns 0-7, 8-15
#pragma unroll
                    for (int n = 0; n < NT; n += 2) {
                        uint32_t vf[4];
                        const int c = n + vc;
                        ldmatrix4_trans(vf, swizzled(vbase + (c >> 3) * (kKeys * 128), vr, c & 7));
                        mma16816<DT>(o[n], high, vf[0], vf[1]);
                        mma16816<DT>(o[n + 1], high, vf[2], vf[3]);
                        mma16816<DT>(o[n], low, vf[0], vf[1]);
                        mma16816<DT>(o[n + 1], low, vf[2], vf[3]);
                    }
                }
            }
            __syncwarp();
            // (a warp that has given up frees nothing: the others may still read the tile)
            if (ok && lane == 0) mbar_arrive(&sh->empty[stage]);
            if (++stage == kStages<D>) {
                stage = 0;
                phase ^= 1;
            }
        }

        // join the four warps: maxima and sums, then the accumulators, warps 0 and 2 first
#pragma unroll
        for (int i = 0; i < 2; ++i) {
#pragma unroll
            for (int w = 0; w < SHARED; ++w) l[i] += __shfl_xor_sync(0xffffffffu, l[i], FIRST << w);
            if ((lane & (((1 << SHARED) - 1) * FIRST)) == 0) {
                sh->m[warp][row_of(i)] = m[i];
                sh->l[warp][row_of(i)] = l[i];
            }
        }
        consumers_sync();
        float f[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int r = row_of(i);
            float top = -INFINITY, sum = 0.0f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) top = fmaxf(top, sh->m[w][r]);
#pragma unroll
            for (int w = 0; w < kWarps; ++w)
                sum += sh->m[w][r] == -INFINITY ? 0.0f : sh->l[w][r] * ex2(sh->m[w][r] - top);
            f[i] = m[i] == -INFINITY ? 0.0f : ex2(m[i] - top);
            if (warp == 0 && (lane & (((1 << SHARED) - 1) * FIRST)) == 0) {   // the barriers of the turns below publish them
                sh->top[r] = top;
                sh->sum[r] = sum;
            }
        }
        float* mine = acc + (warp >> 1) * (ROWS * AS);
#pragma unroll
        for (int turn = 0; turn < 2; ++turn) {
            if ((warp & 1) == turn) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
                    if constexpr (ROWS == 8) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            float* at = mine + (col + (e & 1)) * AS + 16 * n + r0 + 8 * (e >> 1);
                            const float x = o[n][e] * f[e & 1];
                            *at = turn == 1 ? x + *at : x;
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            float2* at = reinterpret_cast<float2*>(mine + (r0 + 8 * i) * AS + 8 * n + col);
                            float2 x = make_float2(o[n][2 * i] * f[i], o[n][2 * i + 1] * f[i]);
                            if (turn == 1) {
                                const float2 y = *at;
                                x.x += y.x;
                                x.y += y.y;
                            }
                            *at = x;
                        }
                    }
            }
            consumers_sync();
        }
        T* op = static_cast<T*>(a.out[rt.rank]) + (size_t)rt.head0 * D;
        auto store_row4 = [&](int r, int d, const float4& x) {
            const int tok = rt.tok0 + r / rt.heads, hd = r % rt.heads;
            const float v[4] = {x.x, x.y, x.z, x.w};
            uint2 w = make_uint2(Payload<DT>::narrow(v), Payload<DT>::narrow(v + 2));
            *reinterpret_cast<uint2*>(op + (size_t)(seg.q.q0 + tok) * a.out_stride + (size_t)hd * D + d) = w;
        };
        float* part = a.partial + (size_t)seg.slot * kPartFloats<ROWS, D>;
        for (int i = tid; i < rt.rows * (D / 4); i += 32 * kWarps) {
            const int r = i / (D / 4), d = i % (D / 4) * 4;
            const float4 x = *reinterpret_cast<const float4*>(acc + r * AS + d);
            const float4 y = *reinterpret_cast<const float4*>(acc + ROWS * AS + r * AS + d);
            float4 z = make_float4(x.x + y.x, x.y + y.y, x.z + y.z, x.w + y.w);
            const float top = sh->top[r], sum = sh->sum[r];
            if (seg.parts == 1) {
                const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
                store_row4(r, d, make_float4(z.x * inv, z.y * inv, z.z * inv, z.w * inv));
            } else {
                __stcg(reinterpret_cast<float4*>(part + r * D + d), z);
                if (d == 0) {
                    __stcg(part + ROWS * D + r, top);
                    __stcg(part + ROWS * D + ROWS + r, sum);
                }
            }
        }
        if (seg.parts > 1) {
            // the barrier orders the other threads' stores before thread 0's release, and the last
            // one's acquire before their loads
            consumers_sync();
            if (tid == 0) {
                unsigned before;
                asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], 1;"
                             : "=r"(before)
                             : "l"(&a.arrived[seg.first_cta])
                             : "memory");
                sh->last = before + 1 == seg.parts;
                if (sh->last) a.arrived[seg.first_cta] = 0;   // for the next call
            }
            consumers_sync();
            if (sh->last) {
                for (int i = tid; i < rt.rows * (D / 4); i += 32 * kWarps) {
                    const int r = i / (D / 4), d = i % (D / 4) * 4;
                    float top = -INFINITY, sum = 0.0f;
                    float4 z = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                    // eight parts at a time, all of their loads in flight at once
                    for (unsigned k0 = 0; k0 < seg.parts; k0 += 8) {
                        float m[8], l[8];
                        float4 x[8];
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            const float* from =
                                a.partial + (size_t)part_slot(seg.first_cta, min(k0 + k, seg.parts - 1)) * kPartFloats<ROWS, D>;
                            m[k] = k0 + k < seg.parts ? __ldcg(from + ROWS * D + r) : -INFINITY;
                            l[k] = __ldcg(from + ROWS * D + ROWS + r);
                            x[k] = __ldcg(reinterpret_cast<const float4*>(from + r * D + d));
                        }
                        float to = top;
#pragma unroll
                        for (int k = 0; k < 8; ++k) to = fmaxf(to, m[k]);
                        const float f = top == -INFINITY ? 0.0f : ex2(top - to);
                        top = to;
                        sum *= f;
                        z = make_float4(z.x * f, z.y * f, z.z * f, z.w * f);
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            const float w = m[k] == -INFINITY ? 0.0f : ex2(m[k] - to);
                            sum = fmaf(l[k], w, sum);
                            z.x = fmaf(x[k].x, w, z.x);
                            z.y = fmaf(x[k].y, w, z.y);
                            z.z = fmaf(x[k].z, w, z.z);
                            z.w = fmaf(x[k].w, w, z.w);
                        }
                    }
                    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
                    store_row4(r, d, make_float4(z.x * inv, z.y * inv, z.z * inv, z.w * inv));
                }
            }
        }
        consumers_sync();   // the buffers are free for the next row tile
    }
}

template <int DT, int D, int ROWS>
__global__ void __launch_bounds__(kTh, kCtas)
attention_decode_kernel(const __grid_constant__ DecodeArgs a, const BatchArgs b, DevStatus* st)
{
    extern __shared__ __align__(1024) uint8_t smem[];
    constexpr int STAGES = kStages<D>;
    float* acc = reinterpret_cast<float*>(smem + STAGES * 2 * kTileBytes<D>);
    DecodeShared* sh = reinterpret_cast<DecodeShared*>(acc + 2 * ROWS * kAccStride<ROWS, D>);
    if (threadIdx.x == 0) {
        for (int i = 0; i < STAGES; ++i) {
            mbar_init(&sh->full[i], 1);
            mbar_init(&sh->empty[i], kWarps);
        }
        mbar_init_fence();
        sh->gave_up = 0;
    }
    // written by the host when the caches were registered: no need to wait for the launch before
    if (threadIdx.x < 2 * a.n) prefetch_map(a.maps + threadIdx.x);
    pdl_acquire_for_copies();
    __syncthreads();   // the ring's barriers are set up
    Cursor cur;
    Seq at;
    const int heads = a.n * a.kv_heads * a.head_groups;
    const bool some = a.few ? split_few<DecodeSplit>(b, a.tm, heads, a.min_units, cur, at, st)
                            : split_work<DecodeSplit, kTh>(b, a.tm, heads, a.min_units, &sh->split, cur, at, st);
    if (!some) {
        pdl_release();
        return;
    }
    if (threadIdx.x >= 32 * kWarps)
        produce<D>(a, b, cur, at, smem, sh, st);
    else
        consume<DT, D, ROWS>(a, b, cur, at, smem, acc, sh, st);
    pdl_release();
}

}  // namespace

size_t attention_decode_partial_floats(const Handle& h, int head_dim)
{
    return (size_t)(2 * kCtas * h.sm_count) * (size_t)(16 * (head_dim + 2));
}

size_t attention_decode_counters(const Handle& h) { return (size_t)(kCtas * h.sm_count); }

int launch_attention_decode(KvCache& kv, const ar_batch_t& b, const AttnCall& c, int window, cudaStream_t s)
{
    Handle& h = *kv.h;
    DecodeArgs a{};
    for (int r = 0; r < h.n; ++r) {
        a.q[r] = c.q[r];
        a.out[r] = c.out[r];
    }
    a.maps = kv.maps;
    a.partial = kv.partial;
    a.arrived = kv.arrived;
    a.q_stride = c.q_stride;
    a.out_stride = c.out_stride;
    a.scale_log2 = c.scale * kLog2e;
    a.n = h.n;
    a.kv_heads = kv.d.kv_heads;
    a.group = c.q_heads / kv.d.kv_heads;
    const DecodeTiles tiles = decode_tiles(a.group, b.max_new);
    const bool eight = tiles.rows == 8;
    a.tile_heads = tiles.heads;
    a.head_groups = tiles.head_groups;
    a.tm = tiles.tokens;
    a.box_tokens = kv.box_tokens;
    a.min_units = 2;
    a.few = b.seqs <= 256 && (b.max_new + a.tm - 1) / a.tm <= 8;
    const uint64_t moved = (uint64_t)h.n * b.tokens * c.q_heads * kv.d.head_dim * 2u * 2u;
    auto run = [&](auto dtc, auto dc, auto rc) -> int {
        constexpr int DT = decltype(dtc)::value, D = decltype(dc)::value, ROWS = decltype(rc)::value;
        static std::atomic<uint32_t> attr_done{0};
        if (!once_per_device(attr_done, [&] {
                return cudaFuncSetAttribute(attention_decode_kernel<DT, D, ROWS>,
                                            cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem<ROWS, D>) == cudaSuccess;
            }))
            return AR_ERR_CUDA;
        rec_begin(h, s);
        const cudaError_t e =
            launch_kernel(h, attention_decode_kernel<DT, D, ROWS>, dim3((unsigned)(kCtas * h.sm_count)), dim3(kTh),
                          kSmem<ROWS, D>, s, a, batch_args(kv, b, window), h.status);
        rec_end(h, s, AR_K_ATTENTION_DECODE, moved);
        return e == cudaSuccess ? launch_status() : AR_ERR_CUDA;
    };
    auto sized = [&](auto dtc, auto dc) -> int {
        return eight ? run(dtc, dc, std::integral_constant<int, 8>{}) : run(dtc, dc, std::integral_constant<int, 16>{});
    };
    using BF = std::integral_constant<int, AR_BF16>;
    using HF = std::integral_constant<int, AR_F16>;
    using D64 = std::integral_constant<int, 64>;
    using D128 = std::integral_constant<int, 128>;
    if (kv.d.dtype == AR_BF16) return kv.d.head_dim == 128 ? sized(BF{}, D128{}) : sized(BF{}, D64{});
    return kv.d.head_dim == 128 ? sized(HF{}, D128{}) : sized(HF{}, D64{});
}

}  // namespace argb
