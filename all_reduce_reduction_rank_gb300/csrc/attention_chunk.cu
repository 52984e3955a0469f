// Paged attention for chunks of new tokens, on the tensor cores (tcgen05).
//
// A row tile is two halves of 128 rows (new tokens x the query heads that
// share a kv head); against it go tiles of 128 keys.  Per key tile and half the
// tensor cores do 4 x 128 x 128 x D flops (1024 cycles for both halves at D =
// 128 and 8192 flops a cycle each way), and the softmax of a half 128 x 128
// exponentials, so the two halves alternate: while one half's softmax runs on
// four warps, the tensor cores do the other half's products.
//
//   warps 0-3, 4-7  softmax of half 0, 1: thread = row.  Scores come from tensor
//                   memory, probabilities go back over them (16 bits, A operand
//                   of the second product), statistics stay in registers
//   warp 8          one thread issues S = Q K^T and O += P V of both halves in turn
//                   (a warp a half let them drift into step: 1364 for 1530 TFLOP/s)
//   warp 9          tensor copies of K and V tiles (pages) into a ring of stages
//   warp 10         tensor copies of the next rows' queries
//   warp 11         waits for the tiles and tells warp 8 together with the probabilities:
//                   issuing a product takes as long as the product, so every wait that
//                   warp 8 does not need shortens the loop
// The last four warps hand registers to the softmax warps, whose threads hold a
// row of 128 scores.  ptxas still spills (112 to 120 bytes a thread; with two parts 132 to
// 196): about 8 loads and 3 stores a warp and key tile, among some 1400 instructions.
//
// Tensor memory (512 columns): S/P of both halves, O of both halves.  Products
// run in the order they are issued, and a half's S of tile j + 1 is issued
// after its P V of tile j: when a softmax warp sees S of j + 1, O holds
// everything up to j and nothing touches it until the warp hands over P, so it
// may rescale O in place without another wait.
//
// Softmax in one pass, base 2, as in the decode kernel: the reference m moves only
// when a row's maximum passes it by far (kSlack, kBelow), so O is rescaled a few times
// at the start of a row and hardly ever later.
//
// Measured on GB300 (n = 8 bf16, heads of 128): 8192 tokens behind 8192 with 64
// query heads 2.08 to 2.24 ms from run to run, 1470 to 1590 TFLOP/s (77 to 83%
// of cuBLAS's burst rate); packed prompts of 4096, 1023, 2501 and 577 tokens with 32
// query heads 200 to 203 us, 985 TFLOP/s.  A key tile of both halves takes about 3000
// cycles, of them 2048 of products: softmax of a half (scores out of tensor memory
// 170, maxima 390, exponentials 950, of which the first half of the keys is already
// being multiplied) and its products follow each other.  A row tile costs about 3
// key tiles more (queries, first scores, last product, output).
//
// Probabilities as one part of the cache's type or as two (AR_OPT_ATTENTION_PARTS): two
// take as many products of the second kind again and the softmax warps' time to make
// them.  8192 tokens on 8192 2.08 / 3.36 ms, packed prompts 199 / 327 us; error against
// 64 bits 1.3 to 1.4 times that of fp32 probabilities / the same (packed prompts bf16
// 2.07e-3 / 1.61e-3).  One is the default: the half step it costs is no more than the
// output's own rounding.
//
// Split of the keys over CTAs: as in the decode kernel (split_work); the parts,
// up to 128 KB each, are joined by a second launch.
#include "paged.cuh"
#include "tmem.cuh"

namespace argb {
namespace {

constexpr int kKeys = 128;
constexpr int kHalf = kAttnTileRows;        // rows of a half
constexpr int kTh = 384;
// Registers a thread: 384 x 168 at launch = 256 x 200 + 128 x 104 (208 / 88: 2% slower,
// 192 / 120: 1%).
constexpr int kSoftmaxRegs = 200, kOtherRegs = 104;

// weight of a row tile's start and end: 2 / 3 / 4 key tiles, packed prompts 208.5 / 204 /
// 203.6 us, 117 tokens on 7752 keys 32.9 / 30.3 / 35.6 us
using ChunkSplit = Split<kKeys, 3, 5>;
using ChunkWalk = Walk<ChunkSplit>;

template <int D> constexpr int kTileBytes = kKeys * D * 2;    // of K, of V, and of a half's Q
template <int D> constexpr int kStages = D == 128 ? 5 : 10;
template <int D> constexpr int kPartFloats = 2 * kHalf * (D + 2);

struct ChunkShared {
    uint64_t full[10], empty[10];
    uint64_t q_full[2], q_empty[2], s_full[2], p_full[2][2], o_full[2], drained;
    SplitShared split;
    uint32_t tmem;
    int gave_up;
    // each warp's place in the run: kept here, so that the loops over the keys
    // have the registers
    ChunkWalk walk[12];
    Segment seg[12];
};
static_assert(sizeof(ChunkShared) <= 3072, "fits beside the tiles");

template <int D> constexpr int kSmem = (2 + kStages<D>) * kTileBytes<D> + 3072;

// Rows whose keys were split: what the join needs, by the CTA of the first part.
struct JoinWork {
    unsigned parts;        // 0 or 1: nothing to join
    int rank, kv_head;
    int row0;              // packed row of the tile's first token
    int rows[2];           // rows of its halves
};

struct ChunkArgs {
    CUtensorMap q[kMaxRanks];                // boxes of a half's tokens and of a kv head's query heads
    void* out[kMaxRanks];
    const CUtensorMap* maps;
    float* partial;
    JoinWork* joins;
    size_t out_stride;
    float scale_log2;
    int n, kv_heads, group;                  // query heads per kv head
    int half_tokens;                         // new tokens of a half: 128 / group
    int box_tokens, min_units;
};

// One half's share of a segment.
struct HalfTile {
    int tok0, rows;    // first new token, rows
    int tiles;         // key tiles of this CTA that it sees any key of
};

__device__ __forceinline__ HalfTile half_tile(const ChunkArgs& a, const Segment& seg, int h)
{
    HalfTile x;
    x.tok0 = (2 * seg.t + h) * a.half_tokens;
    const int tokens = max(min(a.half_tokens, seg.q.nq - x.tok0), 0);
    x.rows = tokens * a.group;
    const int key_hi = tokens ? max(seg.q.c0 + x.tok0 + tokens, 0) : 0;
    x.tiles = max(min((key_hi + kKeys - 1) / kKeys, seg.j1) - seg.j0, 0);
    return x;
}

// The warp's next segment, from and to shared memory.
__device__ __forceinline__ bool next_segment(const BatchArgs& b, int tile_tokens, ChunkShared* sh, DevStatus* st)
{
    const int warp = threadIdx.x / 32;
    ChunkWalk walk = sh->walk[warp];
    Segment seg;
    const bool more = walk.next(b, tile_tokens, seg, st);
    __syncwarp();
    if ((threadIdx.x & 31) == 0) {
        sh->walk[warp] = walk;
        sh->seg[warp] = seg;
    }
    __syncwarp();
    return more;
}

// Waits with the whole warp; false for all its lanes, now and from then on,
// once a wait of the CTA has run out.
__device__ __forceinline__ void warp_wait(bool& ok, uint64_t* bar, uint32_t parity, ChunkShared* sh, DevStatus* st)
{
    if (__all_sync(0xffffffffu, mbar_wait_20us(bar, parity))) return;
    if (ok) ok = wait_on_or_give_up(bar, parity, &sh->gave_up, st);
    ok = __all_sync(0xffffffffu, ok);
}

template <int D>
__device__ void produce(const ChunkArgs& a, const BatchArgs& b, uint8_t* stages, ChunkShared* sh,
                        DevStatus* st)
{
    const int lane = threadIdx.x & 31;
    const int per_tile = kKeys / a.box_tokens;          // boxes of a tile along the keys: 2, 4 or 8
    const int box = lane % per_tile, panel = lane / per_tile;
    const bool mine = panel < D / 64;
    const Segment& seg = sh->seg[threadIdx.x / 32];
    int stage = 0;
    uint32_t phase = 0, issued = 0;
    bool ok = true;
    while (ok && next_segment(b, 2 * a.half_tokens, sh, st)) {
        const int tiles = max(half_tile(a, seg, 0).tiles, half_tile(a, seg, 1).tiles);
        const int kv_head = seg.head % a.kv_heads, rank = seg.head / a.kv_heads;
        if (rank == b.absent) break;
        const int32_t* row = b.table + (size_t)seg.s * b.table_stride;
        const int j0 = seg.j0, key_lo = seg.span.key_lo, key_hi = seg.span.key_hi;
        for (int j = j0; ok && j < j0 + tiles; ++j) {
            const int key = j * kKeys + box * a.box_tokens;
            bool copy = mine && key < key_hi && key + a.box_tokens > key_lo;
            int page = 0;
            if (copy) {
                page = row[key >> b.page_shift];
                if (page < 0 || page >= b.pages) {
                    report_index(st);
                    copy = false;
                }
            }
            const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, copy)) * a.box_tokens * 128u;
            for (int v = 0; v < 2; ++v) {   // K, then V
                if (issued >= (uint32_t)kStages<D>) warp_wait(ok, &sh->empty[stage], phase ^ 1, sh, st);
                if (!ok) break;
                if (lane == 0) mbar_arrive_expect_tx(&sh->full[stage], bytes);
                __syncwarp();
                if (copy)
                    page_copy(stages + (size_t)stage * kTileBytes<D> + panel * (kKeys * 128) + box * a.box_tokens * 128,
                              a.maps + (v ? a.n : 0) + rank, panel * 64, key & ((1 << b.page_shift) - 1), kv_head, page,
                              &sh->full[stage]);
                ++issued;
                if (++stage == kStages<D>) {
                    stage = 0;
                    phase ^= 1;
                }
            }
        }
    }
    wait_for_ring(sh->full, kStages<D>, issued, stage, phase, st);
}

// The halves' queries, as soon as the last product that reads the previous
// ones is done, so that they are there when the softmax warps come from the rows
// before.  A box may reach into the next sequence's tokens or past the last:
// those rows are computed and not written.
template <int D>
__device__ void load_queries(const ChunkArgs& a, const BatchArgs& b, uint8_t* q_tiles, ChunkShared* sh, DevStatus* st)
{
    const int lane = threadIdx.x & 31;
    const Segment& seg = sh->seg[threadIdx.x / 32];
    uint32_t issued[2] = {0, 0};
    bool ok = true;
    while (ok && next_segment(b, 2 * a.half_tokens, sh, st)) {
        const int kv_head = seg.head % a.kv_heads, rank = seg.head / a.kv_heads;
        for (int h = 0; ok && h < 2; ++h) {
            const HalfTile x = half_tile(a, seg, h);
            if (x.tiles == 0) continue;
            if (issued[h] > 0) warp_wait(ok, &sh->q_empty[h], (issued[h] - 1) & 1, sh, st);
            if (!ok) break;
            ++issued[h];
            if (lane == 0) {
                mbar_arrive_expect_tx(&sh->q_full[h], (uint32_t)(a.half_tokens * a.group * D * 2));
                for (int d = 0; d < D; d += 64)
                    box_copy(q_tiles + h * kTileBytes<D> + (d / 64) * (kHalf * 128), &a.q[rank], d, kv_head * a.group,
                             seg.q.q0 + x.tok0, &sh->q_full[h]);
            }
            __syncwarp();
        }
    }
    for (int h = 0; h < 2; ++h)
        if (issued[h] > 0) wait_for_own(&sh->q_full[h], (issued[h] - 1) & 1, st);
}

// The tiles that the products of key tile i read beside the probabilities, V of
// i and K of i + 1: once they are there, the last arrival on the first part's
// barrier of each half that takes part.
template <int D>
__device__ void watch_tiles(const ChunkArgs& a, const BatchArgs& b, uint8_t* stages, ChunkShared* sh, DevStatus* st)
{
    const int lane = threadIdx.x & 31;
    const Segment& seg = sh->seg[threadIdx.x / 32];
    int stage = 0;
    uint32_t phase = 0, p_phase[2] = {0, 0};
    bool ok = true;
    auto step = [&] {
        if (++stage == kStages<D>) {
            stage = 0;
            phase ^= 1;
        }
    };
    while (ok && next_segment(b, 2 * a.half_tokens, sh, st)) {
        const int n[2] = {half_tile(a, seg, 0).tiles, half_tile(a, seg, 1).tiles};
        const int tiles = max(n[0], n[1]), j0 = seg.j0, key_lo = seg.span.key_lo, key_hi = seg.span.key_hi;
        if (tiles == 0) continue;
        step();   // K of the first tile is warp 8's
        for (int i = 0; ok && i < tiles; ++i) {
            const int v_stage = stage;
            warp_wait(ok, &sh->full[stage], phase, sh, st);
            step();
            if (i + 1 < tiles) {
                warp_wait(ok, &sh->full[stage], phase, sh, st);
                step();
            }
            const int key0 = (j0 + i) * kKeys;
            if (key0 + kKeys > key_hi || key0 < key_lo) {
                // slots of these pages that no row sees may hold anything: their values count as 0
                const uint32_t base = smem_addr(stages + v_stage * kTileBytes<D>);
                for (int x = lane; x < kKeys * (D / 8); x += 32) {
                    const int r = x / (D / 8), c = x % (D / 8);
                    if (key0 + r >= key_hi || key0 + r < key_lo) {
                        const uint32_t at = base + (c >> 3) * (kKeys * 128) + r * 128 + (c & 7) * 16;
                        asm volatile("st.shared.v4.b32 [%0], {%1,%1,%1,%1};" ::"r"(at), "r"(0) : "memory");
                    }
                }
                fence_proxy_async();
                __syncwarp();
            }
            for (int h = 0; h < 2; ++h)
                if (i < n[h]) {
                    // one phase at a time: not before the softmax warps' arrivals of the last
                    warp_wait(ok, &sh->p_full[h][0], p_phase[h] ^ 1, sh, st);
                    p_phase[h] ^= 1;
                    // (nothing after giving up: the products would read, and free, tiles that have not landed)
                    if (ok && lane == 0) mbar_arrive(&sh->p_full[h][0]);
                }
        }
    }
}

template <int DT, int D, int PARTS>
__device__ void issue(const ChunkArgs& a, const BatchArgs& b, uint8_t* q_tiles, uint8_t* stages, ChunkShared* sh,
                      DevStatus* st)
{
    constexpr uint32_t kScores = mma_shape(DT == AR_BF16, kKeys, false);
    constexpr uint32_t kValues = mma_shape(DT == AR_BF16, D, true);
    const uint32_t tmem = sh->tmem;
    const Segment& seg = sh->seg[threadIdx.x / 32];
    int stage = 0;                // of the next tile in the ring
    uint32_t phase = 0;
    uint32_t q_phase[2] = {0, 0}, p_phase[2] = {0, 0};
    bool ok = true;
    auto wait = [&](uint64_t* bar, uint32_t parity) { warp_wait(ok, bar, parity, sh, st); };
    auto step = [&](int& s, uint32_t& p) {
        if (++s == kStages<D>) {
            s = 0;
            p ^= 1;
        }
    };
    // S of half h = its Q times the keys in `from`
    auto scores = [&](int h, int from, bool last) {
        if (ok && elect_one()) {
            const uint64_t qa = mma_operand(smem_addr(q_tiles + h * kTileBytes<D>), 1024, 16);
            const uint64_t ka = mma_operand(smem_addr(stages + from * kTileBytes<D>), 1024, 16);
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
                const uint32_t off = ((k / 4) * (kKeys * 128) + (k % 4) * 32) >> 4;
                mma_ss(tmem + h * kKeys, qa + off, ka + off, kScores, k > 0);
            }
            mma_commit(&sh->s_full[h]);
            if (last) mma_commit(&sh->q_empty[h]);
        }
        __syncwarp();
    };
    while (ok && next_segment(b, 2 * a.half_tokens, sh, st)) {
        const int n[2] = {half_tile(a, seg, 0).tiles, half_tile(a, seg, 1).tiles};
        const int tiles = max(n[0], n[1]);
        if (tiles == 0) continue;
        wait(&sh->full[stage], phase);
        for (int h = 0; h < 2; ++h)
            if (n[h] > 0) {
                wait(&sh->q_full[h], q_phase[h]);
                q_phase[h] ^= 1;
                tmem_after_sync();
                scores(h, stage, n[h] == 1);
            }
        if (ok && elect_one()) mma_commit(&sh->empty[stage]);
        __syncwarp();
        step(stage, phase);
        for (int i = 0; ok && i < tiles; ++i) {
            const int v_stage = stage;
            step(stage, phase);
            const int k_stage = stage;
            const bool more = i + 1 < tiles;
            if (more) step(stage, phase);
            for (int h = 0; h < 2; ++h) {
                if (i >= n[h]) continue;
                // the probabilities come in two parts: the product over the first 64 keys runs while
                // the softmax warps do the others
#pragma unroll
                for (int part = 0; part < 2; ++part) {
                    wait(&sh->p_full[h][part], p_phase[h]);
                    tmem_after_sync();
                    if (ok && elect_one()) {
                        const uint64_t va = mma_operand(smem_addr(stages + v_stage * kTileBytes<D>), 1024, kKeys * 128);
#pragma unroll
                        for (int k = 4 * part; k < 4 * part + 4; ++k) {
                            mma_ts(tmem + 2 * kKeys + h * D, tmem + h * kKeys + 8 * k, va + k * (2048 >> 4), kValues,
                                   i > 0 || k > 0);
                            if constexpr (PARTS == 2)
                                mma_ts(tmem + 2 * kKeys + h * D, tmem + h * kKeys + kKeys / 2 + 8 * k,
                                       va + k * (2048 >> 4), kValues, true);
                        }
                        if (part == 1 && i + 1 == n[h]) mma_commit(&sh->o_full[h]);
                    }
                    __syncwarp();
                }
                p_phase[h] ^= 1;
                if (i + 1 < n[h]) scores(h, k_stage, i + 2 == n[h]);
            }
            if (ok && elect_one()) {
                mma_commit(&sh->empty[v_stage]);
                if (more) mma_commit(&sh->empty[k_stage]);
            }
            __syncwarp();
        }
    }
    // nothing that was issued may still run when the tensor memory is freed
    if (elect_one()) mma_commit(&sh->drained);
    __syncwarp();
    wait_for_own(&sh->drained, 0, st);
}

__device__ __forceinline__ uint64_t pack2(float x, float y)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ void unpack2(uint64_t r, float& x, float& y)
{
    asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(r));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b)
{
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

__device__ __forceinline__ float max3(float a, float b, float c)
{
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// Lane i of four consecutive ones holds pieces w[0..3] of row i; after: piece i
// of rows 0..3.
__device__ __forceinline__ void transpose4(uint32_t (&w)[4][4], int lane)
{
#pragma unroll
    for (int d = 1; d < 4; d <<= 1) {
        const bool up = lane & d;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (i & d) continue;
            // swap w[i + d] of the lane without the bit for w[i] of the lane with it
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint32_t give = up ? w[i][k] : w[i + d][k];
                const uint32_t got = __shfl_xor_sync(0xffffffffu, give, d);
                if (up)
                    w[i][k] = got;
                else
                    w[i + d][k] = got;
            }
        }
    }
}

template <int DT, int D, int PARTS>
__device__ void soften(const ChunkArgs& a, const BatchArgs& b, ChunkShared* sh, DevStatus* st)
{
    using T = typename Payload<DT>::scalar_t;
    const int h = threadIdx.x / kHalf, row = threadIdx.x % kHalf, lane = threadIdx.x & 31;
    const uint32_t lanes = (uint32_t)(row & ~31) << 16;
    const uint32_t s_at = sh->tmem + lanes + h * kKeys, o_at = sh->tmem + lanes + 2 * kKeys + h * D;
    bool ok = true;
    uint32_t s_phase = 0, o_phase = 0;

    const int warp = threadIdx.x / 32;
    HalfTile x;
    auto advance = [&] {
        const bool more = next_segment(b, 2 * a.half_tokens, sh, st);
        if (more) x = half_tile(a, sh->seg[warp], h);
        return more;
    };
    bool have = advance();
    while (have) {
        // keys this row sees, and the range that every row of the half sees
        const int first = sh->seg[warp].q.c0 + x.tok0, j0 = sh->seg[warp].j0, tiles = x.tiles;
        const int limit = row < x.rows ? first + row / a.group + 1 : 0;
        const int lower = b.window > 0 ? limit - b.window : 0;
        const int all_hi = first + 1;
        const int all_lo = b.window > 0 ? first + x.rows / a.group - b.window : 0;
        float m = -INFINITY;
        uint64_t l2[2] = {0ull, 0ull};
        float l_before = 0.0f;   // the sum before the last move of m
        for (int i = 0; i < tiles; ++i) {
            warp_wait(ok, &sh->s_full[h], s_phase, sh, st);
            s_phase ^= 1;
            if (!ok) break;
            tmem_after_sync();
            float s[kKeys];
#pragma unroll
            for (int k = 0; k < kKeys; k += 32) tmem_ld32(s + k, s_at + k);
            tmem_wait_ld();
            const int key0 = (j0 + i) * kKeys;
            if (key0 + kKeys > all_hi || key0 < all_lo) {
                const int hi = limit - key0, lo = lower - key0;
#pragma unroll
                for (int k = 0; k < kKeys; ++k)
                    if (k >= hi || k < lo) s[k] = -INFINITY;
            }
            float mx[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
            for (int k = 4; k + 8 <= kKeys; k += 8)
#pragma unroll
                for (int e = 0; e < 4; ++e) mx[e] = max3(mx[e], s[k + e], s[k + 4 + e]);
#pragma unroll
            for (int e = 0; e < 4; ++e) mx[e] = fmaxf(mx[e], s[kKeys - 4 + e]);
            const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * a.scale_log2;
            const bool move = top > m + (kSlack + kBelow<DT>);
            const bool rescale = __any_sync(0xffffffffu, move);
            float f = 1.0f;
            if (rescale) {
                const float to = move ? top - kBelow<DT> : m;
                f = m == -INFINITY ? 0.0f : ex2(m - to);
                m = to;
                float p, q, u, v;
                unpack2(l2[0], p, q);
                unpack2(l2[1], u, v);
                l_before = (l_before + ((p + q) + (u + v))) * f;
                l2[0] = l2[1] = 0ull;
            }
            if (rescale && i > 0) {
#pragma unroll 1
                for (int k = 0; k < D; k += 16) {
                    float o[16];
                    tmem_ld16(o, o_at + k);
                    tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 16; ++e) o[e] *= f;
                    tmem_st16(o_at + k, reinterpret_cast<const uint32_t*>(o));
                }
            }
            const float ref = m == -INFINITY ? 0.0f : m;
            const uint64_t sc = pack2(a.scale_log2, a.scale_log2), off = pack2(-ref, -ref);
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                uint32_t pw[16], rest[16];
#pragma unroll
                for (int k = 0; k < 16; ++k) {
                    float y[2];
                    const int e = 32 * g + 2 * k;
                    unpack2(fma2(pack2(s[e], s[e + 1]), sc, off), y[0], y[1]);
                    y[0] = ex2(y[0]);
                    y[1] = ex2(y[1]);
                    l2[k & 1] = add2(l2[k & 1], pack2(y[0], y[1]));
                    // the product's operand has the cache's type: p rounded to it (at most half a step of it
                    // each), and with two parts what that left out, in the other half of the scores' place
                    pw[k] = Payload<DT>::narrow(y);
                    if constexpr (PARTS == 2) {
                        float back[2];
                        Payload<DT>::widen(pw[k], back);
                        back[0] = y[0] - back[0];
                        back[1] = y[1] - back[1];
                        rest[k] = Payload<DT>::narrow(back);
                    }
                }
                tmem_st16(s_at + 16 * g, pw);
                if constexpr (PARTS == 2) tmem_st16(s_at + kKeys / 2 + 16 * g, rest);
                if (g & 1) {
                    tmem_wait_st();
                    tmem_before_sync();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sh->p_full[h][g / 2]);
                }
            }
        }
        const Segment seg = sh->seg[warp];
        const HalfTile done = x;
        have = advance();

        // the row's sum and result
        float p, q, u, v;
        unpack2(l2[0], p, q);
        unpack2(l2[1], u, v);
        const float l = l_before + ((p + q) + (u + v));
        if (done.tiles > 0) {
            warp_wait(ok, &sh->o_full[h], o_phase, sh, st);
            o_phase ^= 1;
            tmem_after_sync();
        }
        const int kv_head = seg.head % a.kv_heads, rank = seg.head / a.kv_heads;
        // 32 columns of the warp's rows: four lanes swap their 16-byte pieces, so that a store
        // writes 64 bytes of 8 rows, not 16 of 32
        T* to[4];
        bool there[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int r = (row & ~3) + k;
            there[k] = r < done.rows && ok;
            to[k] = static_cast<T*>(a.out[rank]) + (size_t)(seg.q.q0 + done.tok0 + r / a.group) * a.out_stride +
                    (size_t)(kv_head * a.group + r % a.group) * D + 8 * (row & 3);
        }
        auto store32 = [&](const float* o, int k) {
            uint32_t w[4][4];
#pragma unroll
            for (int e = 0; e < 16; ++e) w[e / 4][e % 4] = Payload<DT>::narrow(o + 2 * e);
            transpose4(w, lane);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (there[e]) st16_next(to[e] + k, make_uint4(w[e][0], w[e][1], w[e][2], w[e][3]));
        };
        if (seg.parts == 1) {
            const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll 1
            for (int k = 0; k < D; k += 32) {
                float o[32];
                if (done.tiles > 0 && ok) {
                    tmem_ld32(o, o_at + k);
                    tmem_wait_ld();
                }
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = done.tiles > 0 ? o[e] * inv : 0.0f;
                store32(o, k);
            }
        } else {
            // column after column, so that the warp's rows are consecutive words
            float* part = a.partial + (size_t)seg.slot * kPartFloats<D> + h * (kHalf * (D + 2));
            if (done.tiles > 0 && ok)
#pragma unroll 1
                for (int k = 0; k < D; k += 32) {
                    float o[32];
                    tmem_ld32(o, o_at + k);
                    tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 32; ++e) __stcg(part + (k + e) * kHalf + row, o[e]);
                }
            // NaN scores never move m.  Where all are NaN it would still say that the part saw nothing,
            // and the row would not come out as NaN as it does when it is not split
            __stcg(part + D * kHalf + row, l != l ? 0.0f : m);
            __stcg(part + (D + 1) * kHalf + row, l);
            if (seg.slot & 1) {   // the first part
                if (row == 0) {
                    JoinWork& j = a.joins[blockIdx.x];
                    if (h == 0) {
                        j.rank = rank;
                        j.kv_head = kv_head;
                        j.row0 = seg.q.q0 + done.tok0;
                        j.parts = seg.parts;
                    }
                    j.rows[h] = done.rows;
                }
            }
        }
    }
}

template <int DT, int D, int PARTS>
__global__ void __launch_bounds__(kTh, 1)
attention_chunk_kernel(const __grid_constant__ ChunkArgs a, const BatchArgs b, DevStatus* st)
{
    extern __shared__ __align__(1024) uint8_t smem[];
    uint8_t* q_tiles = smem;
    uint8_t* stages = smem + 2 * kTileBytes<D>;
    ChunkShared* sh = reinterpret_cast<ChunkShared*>(stages + kStages<D> * kTileBytes<D>);
    const int warp = threadIdx.x / 32;
    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages<D>; ++i) {
            mbar_init(&sh->full[i], 1);
            mbar_init(&sh->empty[i], 1);
        }
        for (int h = 0; h < 2; ++h) {
            mbar_init(&sh->q_full[h], 1);
            mbar_init(&sh->q_empty[h], 1);
            mbar_init(&sh->s_full[h], 1);
            mbar_init(&sh->p_full[h][0], kHalf / 32 + 1);
            mbar_init(&sh->p_full[h][1], kHalf / 32);
            mbar_init(&sh->o_full[h], 1);
        }
        mbar_init(&sh->drained, 1);
        mbar_init_fence();
        sh->gave_up = 0;
    }
    // written by the host when the caches were registered: no need to wait for the launch before
    if (threadIdx.x < 2 * a.n) prefetch_map(a.maps + threadIdx.x);
    pdl_acquire_for_copies();
    if (threadIdx.x == 0) a.joins[blockIdx.x].parts = 0;
    Cursor cur;
    Seq at;
    if (!split_work<ChunkSplit, kTh>(b, 2 * a.half_tokens, a.n * a.kv_heads, a.min_units, &sh->split, cur, at, st)) {
        pdl_release();
        return;
    }
    if (threadIdx.x % 32 == 0) sh->walk[warp] = ChunkWalk(cur, at);
    if (warp == 8) tmem_alloc(&sh->tmem, 512);
    tmem_before_sync();
    __syncthreads();
    tmem_after_sync();
    if (warp < 8) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
        soften<DT, D, PARTS>(a, b, sh, st);
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
        if (warp == 8)
            issue<DT, D, PARTS>(a, b, q_tiles, stages, sh, st);
        else if (warp == 9)
            produce<D>(a, b, stages, sh, st);
        else if (warp == 10)
            load_queries<D>(a, b, q_tiles, sh, st);
        else
            watch_tiles<D>(a, b, stages, sh, st);
    }
    pdl_release();
    tmem_before_sync();
    __syncthreads();
    if (warp == 8) {
        tmem_after_sync();
        tmem_free(sh->tmem, 512);
    }
}

// Joins the parts of the rows whose keys were split, in the order of the keys:
// o = sum 2^(m_k - m) o_k / sum 2^(m_k - m) l_k.  A launch of its own, so that
// every SM takes a share of what one CTA of the first launch would read alone;
// a block takes 16 columns of a half's 128 rows.
constexpr int kJoinColumns = 16;

template <int DT, int D>
__global__ void __launch_bounds__(kHalf)
attention_join_kernel(const __grid_constant__ ChunkArgs a)
{
    using T = typename Payload<DT>::scalar_t;
    pdl_acquire();
    pdl_release();
    const unsigned f = blockIdx.x;
    const int h = blockIdx.y / (D / kJoinColumns), d = blockIdx.y % (D / kJoinColumns) * kJoinColumns;
    const JoinWork j = a.joins[f];
    const int row = threadIdx.x;
    if (j.parts < 2 || row >= j.rows[h]) return;
    auto part_of = [&](unsigned k) {
        return a.partial + (size_t)part_slot(f, k) * kPartFloats<D> + h * (kHalf * (D + 2)) + row;
    };
    // four parts at a time, all of their loads in flight at once; a later part with a larger
    // maximum scales what is there
    float top = -INFINITY, o[kJoinColumns], sum = 0.0f;
#pragma unroll
    for (int e = 0; e < kJoinColumns; ++e) o[e] = 0.0f;
    for (unsigned k0 = 0; k0 < j.parts; k0 += 4) {
        float m[4], l[4], x[4][kJoinColumns];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float* from = part_of(min(k0 + k, j.parts - 1));
            m[k] = k0 + k < j.parts ? __ldcg(from + D * kHalf) : -INFINITY;
            l[k] = __ldcg(from + (D + 1) * kHalf);
#pragma unroll
            for (int e = 0; e < kJoinColumns; ++e) x[k][e] = __ldcg(from + (d + e) * kHalf);
        }
        const float to = fmaxf(top, fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3])));
        const float f = top == -INFINITY ? 0.0f : ex2(top - to);
        top = to;
        sum *= f;
#pragma unroll
        for (int e = 0; e < kJoinColumns; ++e) o[e] *= f;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            // a part that saw nothing wrote no columns: whatever is there does not count
            const bool saw = m[k] != -INFINITY;
            const float w = saw ? ex2(m[k] - to) : 0.0f;
            sum = fmaf(saw ? l[k] : 0.0f, w, sum);
#pragma unroll
            for (int e = 0; e < kJoinColumns; ++e) o[e] = fmaf(saw ? x[k][e] : 0.0f, w, o[e]);
        }
    }
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    const int r = row + h * a.half_tokens * a.group;   // rows of half 0 come first
    T* to = static_cast<T*>(a.out[j.rank]) + (size_t)(j.row0 + r / a.group) * a.out_stride +
            (size_t)(j.kv_head * a.group + r % a.group) * D + d;
#pragma unroll
    for (int e = 0; e < kJoinColumns; ++e) o[e] *= inv;
#pragma unroll
    for (int e = 0; e < kJoinColumns; e += 8) st16_next(to + e, round_vec<DT>(o + e));
}

}  // namespace

size_t attention_chunk_partial_floats(const Handle& h, int head_dim)
{
    return (size_t)(2 * h.sm_count) * (size_t)(2 * kHalf * (head_dim + 2));
}

size_t attention_chunk_join_bytes(const Handle& h) { return (size_t)h.sm_count * sizeof(JoinWork); }

int launch_attention_chunk(KvCache& kv, const ar_batch_t& b, const AttnCall& c, int window, cudaStream_t s)
{
    Handle& h = *kv.h;
    ChunkArgs a{};
    const int group = c.q_heads / kv.d.kv_heads;
    for (int r = 0; r < h.n; ++r) {
        const size_t dims[3] = {(size_t)kv.d.head_dim, (size_t)c.q_heads, b.tokens};
        const size_t strides[2] = {(size_t)kv.d.head_dim * 2, c.q_stride * 2};
        const unsigned box[3] = {64, (unsigned)group, (unsigned)(kHalf / group)};
        if (int rc = encode_map(kv, &a.q[r], 3, c.q[r], dims, strides, box)) return rc;
        a.out[r] = c.out[r];
    }
    a.maps = kv.maps;
    a.partial = kv.partial;
    a.joins = static_cast<JoinWork*>(kv.joins);
    a.out_stride = c.out_stride;
    a.scale_log2 = c.scale * kLog2e;
    a.n = h.n;
    a.kv_heads = kv.d.kv_heads;
    a.group = group;
    a.half_tokens = kHalf / a.group;
    a.box_tokens = kv.box_tokens;
    a.min_units = 4;
    const uint64_t moved = (uint64_t)h.n * b.tokens * c.q_heads * kv.d.head_dim * 2u * 2u;
    auto run = [&](auto dtc, auto dc, auto pc) -> int {
        constexpr int DT = decltype(dtc)::value, D = decltype(dc)::value, PARTS = decltype(pc)::value;
        static std::atomic<uint32_t> attr_done{0};
        if (!once_per_device(attr_done, [&] {
                return cudaFuncSetAttribute(attention_chunk_kernel<DT, D, PARTS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                            kSmem<D>) == cudaSuccess;
            }))
            return AR_ERR_CUDA;
        rec_begin(h, s);
        const cudaError_t e = launch_kernel(h, attention_chunk_kernel<DT, D, PARTS>, dim3((unsigned)h.sm_count), dim3(kTh),
                                            kSmem<D>, s, a, batch_args(kv, b, window), h.status);
        const cudaError_t e2 = launch_kernel(h, attention_join_kernel<DT, D>,
                                             dim3((unsigned)h.sm_count, 2 * D / kJoinColumns), dim3(kHalf), 0, s, a);
        rec_end(h, s, AR_K_ATTENTION_CHUNK, moved, 2);
        return e == cudaSuccess && e2 == cudaSuccess ? launch_status() : AR_ERR_CUDA;
    };
    auto parts = [&](auto dtc, auto dc) -> int {
        return h.attention_parts == 2 ? run(dtc, dc, std::integral_constant<int, 2>{})
                                      : run(dtc, dc, std::integral_constant<int, 1>{});
    };
    using BF = std::integral_constant<int, AR_BF16>;
    using HF = std::integral_constant<int, AR_F16>;
    using D64 = std::integral_constant<int, 64>;
    using D128 = std::integral_constant<int, 128>;
    if (kv.d.dtype == AR_BF16) return kv.d.head_dim == 128 ? parts(BF{}, D128{}) : parts(BF{}, D64{});
    return kv.d.head_dim == 128 ? parts(HF{}, D128{}) : parts(HF{}, D64{});
}

}  // namespace argb
