// C-ABI entry points of the paged caches, the rotation and append, and the
// attention (declared in include/ar.h): argument checks and launches.  Host
// code only; nothing here allocates after ar_kv_create.
#include <algorithm>
#include <climits>
#include <cmath>
#include <cstring>
#include <new>
#include <utility>

#include <cudaTypedefs.h>

#include "common.cuh"
#include "layer.h"

using namespace argb;

namespace {

constexpr uint32_t kKvMagic = 0x41524b56u;  // "ARKV"

constexpr size_t kMaxStride = (size_t)1 << 39;   // elements: tensor copies take strides below 2^40 bytes

int check_desc(const ar_kv_desc_t* d)
{
    if (!d) return AR_ERR_INVALID;
    if (d->dtype != AR_BF16 && d->dtype != AR_F16) return AR_ERR_INVALID;
    if (d->kv_heads < 1 || d->kv_heads > 1024) return AR_ERR_INVALID;
    if (d->head_dim != 64 && d->head_dim != 128) return AR_ERR_INVALID;
    if (d->page_size != 16 && d->page_size != 32 && d->page_size != 64 && d->page_size != 128) return AR_ERR_INVALID;
    if (d->pages < 1 || d->pages > (size_t)INT_MAX) return AR_ERR_INVALID;
    for (size_t st : {d->page_stride, d->head_stride, d->token_stride})
        if (st == 0 || st % 8 != 0 || st >= kMaxStride) return AR_ERR_INVALID;
    if (d->token_stride < (size_t)d->head_dim) return AR_ERR_INVALID;
    // page * page_stride fits 64 bits by far (no address space has 2^59 bytes)
    if (d->pages - 1 > ((size_t)1 << 58) / d->page_stride) return AR_ERR_INVALID;
    return AR_OK;
}

int check_batch(const ar_batch_t* b)
{
    if (!b) return AR_ERR_INVALID;
    // the kernels look a little past the last sequence in 32 bits before they compare
    if (b->seqs < 0 || b->seqs > 1 << 30 || b->tokens > (size_t)1 << 30) return AR_ERR_INVALID;
    if (b->tokens == 0) return AR_OK;
    if (b->seqs == 0 || b->max_new < 1) return AR_ERR_INVALID;
    if (!b->q_start || !b->kv_len || !b->page_table) return AR_ERR_INVALID;
    if (((uintptr_t)b->q_start | (uintptr_t)b->kv_len | (uintptr_t)b->page_table) & 3u) return AR_ERR_ALIGN;
    if (b->table_stride == 0 || b->table_stride > (size_t)1 << 27) return AR_ERR_INVALID;
    return AR_OK;
}

// n pointers to rows of `heads` heads, `stride` elements apart.
int check_rows(int n, const void* const* p, size_t row, size_t stride, size_t tokens)
{
    if (!p) return AR_ERR_INVALID;
    for (int r = 0; r < n; ++r)
        if (!p[r]) return AR_ERR_INVALID;
    if (stride < row || stride % 8 != 0 || stride >= kMaxStride || stride > ((size_t)1 << 40) / (tokens ? tokens : 1))
        return AR_ERR_INVALID;
    for (int r = 0; r < n; ++r)
        if (!aligned16(p[r])) return AR_ERR_ALIGN;
    return AR_OK;
}

// Rows of 16-bit elements a (an x row ea, sa apart) meet rows b.  Slices of one
// allocation whose rows interleave (equal strides, disjoint columns) do not.
bool rows_overlap(const void* a, size_t ea, size_t sa, const void* b, size_t eb, size_t sb, size_t tokens)
{
    if (!tokens) return false;
    const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
    const size_t xn = ((tokens - 1) * sa + ea) * 2, yn = ((tokens - 1) * sb + eb) * 2;
    if (x >= y + yn || y >= x + xn) return false;
    if (sa != sb) return true;
    const size_t s = sa * 2, at = x >= y ? (x - y) % s : (s - (y - x) % s) % s;   // a's place in b's rows
    return at < eb * 2 || at + ea * 2 > s;
}

// `count` blocks of `width` bytes, `stride` apart.
struct Blocks {
    uintptr_t at;
    size_t width, stride, count;
    uintptr_t end() const { return at + (count - 1) * stride + width; }
};

// Some block of a and some block of b share a byte.
bool blocks_meet(Blocks a, Blocks b)
{
    if (a.count > b.count) std::swap(a, b);
    for (size_t i = 0; i < a.count; ++i) {
        const uintptr_t lo = a.at + i * a.stride, hi = lo + a.width;
        if (hi <= b.at) continue;
        const size_t j = std::min((size_t)(hi - 1 - b.at) / b.stride, b.count - 1);   // the last that begins before hi
        if (b.at + j * b.stride + b.width > lo) return true;
    }
    return false;
}

// The caches' pages and n buffers of rows.  A page counts with what lies between
// its slots and heads.
int check_apart(int n, const ar_kv_desc_t& d, void* const* k, void* const* v, const void* const* rows, size_t row,
                size_t stride, size_t tokens)
{
    if (tokens == 0) return AR_OK;
    const size_t page = ((size_t)d.kv_heads - 1) * d.head_stride + ((size_t)d.page_size - 1) * d.token_stride +
                        (size_t)d.head_dim;
    const size_t length = Blocks{0, 2 * page, 2 * d.page_stride, d.pages}.end();
    for (int r = 0; r < n; ++r) {
        const Blocks x{(uintptr_t)rows[r], 2 * row, 2 * stride, tokens};
        const uintptr_t lo = x.at, hi = x.end();
        for (int c = 0; c < 2 * n; ++c) {
            const uintptr_t at = (uintptr_t)(c < n ? k[c] : v[c - n]);
            if (lo >= at + length || at >= hi) continue;   // buffers that lie apart, as usual
            if (blocks_meet(x, Blocks{at, 2 * page, 2 * d.page_stride, d.pages})) return AR_ERR_INVALID;
        }
    }
    return AR_OK;
}

// Some slot of the cache at a shares an element with one of the cache at b (the same
// cache: with another of its slots).  Both have the description's strides: the
// places differ by dp pages, dh heads and dt slots, and for every dh and dt the dp
// that come near are two.
bool slots_meet(const ar_kv_desc_t& d, const void* a, const void* b)
{
    const int64_t D = d.head_dim, ps = (int64_t)d.page_stride, pages = (int64_t)d.pages;
    const int64_t apart = ((int64_t)(uintptr_t)a - (int64_t)(uintptr_t)b) / 2;   // elements; both 16-byte aligned
    const int64_t page = ((int64_t)d.kv_heads - 1) * (int64_t)d.head_stride +
                         ((int64_t)d.page_size - 1) * (int64_t)d.token_stride + D;
    const int64_t length = (pages - 1) * ps + page;
    if (apart >= length || -apart >= length) return false;
    for (int dh = 1 - d.kv_heads; dh < d.kv_heads; ++dh)
        for (int dt = 1 - d.page_size; dt < d.page_size; ++dt) {
            const int64_t r = apart + dh * (int64_t)d.head_stride + dt * (int64_t)d.token_stride;
            const int64_t below = r / ps - (r % ps < 0 ? 1 : 0);
            for (int64_t dp = below; dp <= below + 1; ++dp)
                if (dp > -pages && dp < pages && r - dp * ps < D && dp * ps - r < D &&
                    !(a == b && dh == 0 && dt == 0 && dp == 0))
                    return true;
        }
    return false;
}

int check_kv(int n, const ar_kv_desc_t* d, void* const* k, void* const* v)
{
    if (n < 2 || n > kMaxRanks) return AR_ERR_INVALID;
    if (int rc = check_desc(d)) return rc;
    if (!k || !v) return AR_ERR_INVALID;
    for (int r = 0; r < n; ++r)
        if (!k[r] || !v[r]) return AR_ERR_INVALID;
    for (int r = 0; r < n; ++r)
        if (!aligned16(k[r]) || !aligned16(v[r])) return AR_ERR_ALIGN;
    if (slots_meet(*d, k[0], k[0])) return AR_ERR_INVALID;
    const auto cache = [&](int c) { return c < n ? k[c] : v[c - n]; };
    for (int c = 0; c < 2 * n; ++c)
        for (int e = 0; e < c; ++e)
            if (cache(c) == cache(e) || slots_meet(*d, cache(c), cache(e))) return AR_ERR_INVALID;
    return AR_OK;
}

int check_rope(int n, const ar_kv_desc_t& d, const ar_batch_t* b, const RopeCall& c)
{
    const size_t D = (size_t)d.head_dim, krow = D * (size_t)d.kv_heads;
    if (int rc = check_batch(b)) return rc;
    if (c.rot_dim < 0 || c.rot_dim % 16 != 0 || c.rot_dim > (int)D) return AR_ERR_INVALID;
    if (c.interleaved != 0 && c.interleaved != 1) return AR_ERR_INVALID;
    if (c.rot_dim > 0 && (!c.cos_sin || c.max_positions == 0 || c.max_positions > (size_t)1 << 40))
        return AR_ERR_INVALID;
    if (c.rot_dim > 0 && !aligned16(c.cos_sin)) return AR_ERR_ALIGN;
    if ((c.q == nullptr) != (c.q_out == nullptr)) return AR_ERR_INVALID;
    if (int rc = check_rows(n, c.k, krow, c.kv_stride, b->tokens)) return rc;
    if (int rc = check_rows(n, c.v, krow, c.kv_stride, b->tokens)) return rc;
    if (!c.q) return AR_OK;
    if (c.q_heads < 1 || c.q_heads > 65536) return AR_ERR_INVALID;
    const size_t qrow = D * (size_t)c.q_heads;
    if (int rc = check_rows(n, c.q, qrow, c.q_stride, b->tokens)) return rc;
    if (int rc = check_rows(n, c.q_out, qrow, c.q_out_stride, b->tokens)) return rc;
    for (int r = 0; r < n; ++r)
        for (int o = 0; o < n; ++o) {
            const bool same = o == r && c.q_out[r] == c.q[o] && c.q_out_stride == c.q_stride;
            if (!same && rows_overlap(c.q_out[r], qrow, c.q_out_stride, c.q[o], qrow, c.q_stride, b->tokens))
                return AR_ERR_INVALID;
            if (rows_overlap(c.q_out[r], qrow, c.q_out_stride, c.k[o], krow, c.kv_stride, b->tokens) ||
                rows_overlap(c.q_out[r], qrow, c.q_out_stride, c.v[o], krow, c.kv_stride, b->tokens) ||
                (o != r && rows_overlap(c.q_out[r], qrow, c.q_out_stride, c.q_out[o], qrow, c.q_out_stride, b->tokens)))
                return AR_ERR_INVALID;
        }
    return AR_OK;
}

int check_attention(int n, const ar_kv_desc_t& d, const ar_batch_t* b, const AttnCall& c, int window)
{
    if (int rc = check_batch(b)) return rc;
    if (c.q_heads < 1 || c.q_heads % d.kv_heads != 0 || c.q_heads / d.kv_heads > kMaxGroup) return AR_ERR_INVALID;
    if (!(c.scale > 0.0f) || !std::isfinite(c.scale * kLog2e) || window < 0) return AR_ERR_INVALID;
    const size_t row = (size_t)d.head_dim * (size_t)c.q_heads;
    if (int rc = check_rows(n, c.q, row, c.q_stride, b->tokens)) return rc;
    if (int rc = check_rows(n, c.out, row, c.out_stride, b->tokens)) return rc;
    for (int r = 0; r < n; ++r)
        for (int o = 0; o < n; ++o)
            if (rows_overlap(c.out[r], row, c.out_stride, c.q[o], row, c.q_stride, b->tokens) ||
                (o != r && rows_overlap(c.out[r], row, c.out_stride, c.out[o], row, c.out_stride, b->tokens)))
                return AR_ERR_INVALID;
    return AR_OK;
}

}  // namespace

int argb::encode_map(const KvCache& kv, CUtensorMap* map, int dims, const void* base, const size_t* size,
                     const size_t* strides, const unsigned* box)
{
    cuuint64_t sz[5], st[5];
    cuuint32_t bx[5], ones[5];
    for (int i = 0; i < dims; ++i) {
        sz[i] = size[i];
        if (i > 0) st[i - 1] = strides[i - 1];
        bx[i] = box[i];
        ones[i] = 1;
    }
    const auto type = kv.d.dtype == AR_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    const CUresult rc = ((PFN_cuTensorMapEncodeTiled_v12000)kv.encode)(
        map, type, (cuuint32_t)dims, const_cast<void*>(base), sz, st, bx, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
        CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return rc == CUDA_SUCCESS ? AR_OK : AR_ERR_INVALID;
}

struct ar_kv_ctx {
    uint32_t magic;
    KvCache kv;
};

static KvCache* get(ar_kv k) { return k && k->magic == kKvMagic ? &k->kv : nullptr; }

static void note(Handle& h, int op, size_t count, uint64_t rd, uint64_t wr, cudaStream_t s)
{
    std::memset(&h.last, 0, sizeof(h.last));
    h.last.op = op;
    h.last.n_ranks = h.n;
    h.last.count = count;
    h.last.elem_bytes = 2;
    h.last.launches = count ? 1 : 0;
    h.last.hbm_read_bytes = rd;
    h.last.hbm_write_bytes = wr;
    h.last_stream = s;
}

extern "C" {

int ar_kv_create(ar_handle hd, const ar_kv_desc_t* d, void* const* k, void* const* v, ar_kv* out)
{
    Handle* h = handle_of(hd);
    if (!h || !out) return AR_ERR_INVALID;
    if (int rc = check_kv(h->n, d, k, v)) return rc;
    ar_kv_ctx* c = new (std::nothrow) ar_kv_ctx();
    if (!c) return AR_ERR_INVALID;
    KvCache& kv = c->kv;
    kv.h = h;
    kv.d = *d;
    kv.box_tokens = d->page_size < 64 ? d->page_size : 64;
    for (int r = 0; r < h->n; ++r) {
        kv.k[r] = k[r];
        kv.v[r] = v[r];
    }
    const int rc = on_device(*h, [&]() -> int {
        void* fn = nullptr;
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &found) !=
                cudaSuccess ||
            found != cudaDriverEntryPointSuccess || !fn)
            return AR_ERR_CUDA;
        kv.encode = fn;
        alignas(64) CUtensorMap maps[2 * kMaxRanks];
        const size_t size[4] = {(size_t)d->head_dim, (size_t)d->page_size, (size_t)d->kv_heads, d->pages};
        const size_t strides[3] = {d->token_stride * 2, d->head_stride * 2, d->page_stride * 2};
        const unsigned box[4] = {64, (unsigned)kv.box_tokens, 1, 1};
        for (int r = 0; r < h->n; ++r)
            if (encode_map(kv, &maps[r], 4, k[r], size, strides, box) != AR_OK ||
                encode_map(kv, &maps[h->n + r], 4, v[r], size, strides, box) != AR_OK)
                return AR_ERR_INVALID;
        const size_t floats = std::max(attention_decode_partial_floats(*h, d->head_dim),
                                       attention_chunk_partial_floats(*h, d->head_dim));
        const size_t counters = attention_decode_counters(*h), join_bytes = attention_chunk_join_bytes(*h);
        const size_t map_bytes = 2u * (size_t)h->n * sizeof(CUtensorMap);
        if (cudaMalloc(&kv.maps, map_bytes) != cudaSuccess || cudaMalloc(&kv.partial, floats * 4u) != cudaSuccess ||
            cudaMalloc(&kv.arrived, counters * sizeof(unsigned)) != cudaSuccess ||
            cudaMalloc(&kv.joins, join_bytes) != cudaSuccess ||
            cudaMemcpy(kv.maps, maps, map_bytes, cudaMemcpyHostToDevice) != cudaSuccess ||
            cudaMemset(kv.arrived, 0, counters * sizeof(unsigned)) != cudaSuccess ||
            cudaDeviceSynchronize() != cudaSuccess) {
            cudaGetLastError();
            if (kv.maps) cudaFree(kv.maps);
            if (kv.partial) cudaFree(kv.partial);
            if (kv.arrived) cudaFree(kv.arrived);
            if (kv.joins) cudaFree(kv.joins);
            return AR_ERR_CUDA;
        }
        return AR_OK;
    });
    if (rc != AR_OK) {
        delete c;
        return rc;
    }
    c->magic = kKvMagic;
    *out = c;
    return AR_OK;
}

int ar_check_kv(int n_ranks, const ar_kv_desc_t* desc, void* const* k, void* const* v)
{
    return check_kv(n_ranks, desc, k, v);
}

int ar_check_rows_apart(int n_ranks, const ar_kv_desc_t* desc, void* const* k, void* const* v,
                        const void* const* rows, size_t row, size_t stride, size_t tokens)
{
    if (int rc = check_kv(n_ranks, desc, k, v)) return rc;
    if (int rc = check_rows(n_ranks, rows, row, stride, tokens)) return rc;
    return check_apart(n_ranks, *desc, k, v, rows, row, stride, tokens);
}

int ar_check_rope_append(int n_ranks, const ar_kv_desc_t* desc, const ar_batch_t* b, const void* const* q,
                         const void* const* k, const void* const* v, void* const* q_out, int q_heads, size_t q_stride,
                         size_t kv_stride, size_t q_out_stride, const float* cos_sin, size_t max_positions,
                         int rot_dim, int interleaved)
{
    if (n_ranks < 2 || n_ranks > kMaxRanks) return AR_ERR_INVALID;
    if (int rc = check_desc(desc)) return rc;
    return check_rope(n_ranks, *desc, b, RopeCall{q, k, v, q_out, q_heads, q_stride, kv_stride, q_out_stride, cos_sin,
                                                  max_positions, rot_dim, interleaved});
}

int ar_check_paged_attention(int n_ranks, const ar_kv_desc_t* desc, const ar_batch_t* b, const void* const* q,
                             void* const* out, int q_heads, size_t q_stride, size_t out_stride, float scale,
                             int window)
{
    if (n_ranks < 2 || n_ranks > kMaxRanks) return AR_ERR_INVALID;
    if (int rc = check_desc(desc)) return rc;
    return check_attention(n_ranks, *desc, b, AttnCall{q, out, q_heads, q_stride, out_stride, scale}, window);
}

int ar_kv_destroy(ar_kv k)
{
    KvCache* kv = get(k);
    if (!kv) return AR_ERR_INVALID;
    const int rc = on_device(*kv->h, [&] {
        int r = cudaDeviceSynchronize() == cudaSuccess ? AR_OK : AR_ERR_CUDA;
        if (cudaFree(kv->maps) != cudaSuccess) r = AR_ERR_CUDA;
        if (cudaFree(kv->partial) != cudaSuccess) r = AR_ERR_CUDA;
        if (cudaFree(kv->arrived) != cudaSuccess) r = AR_ERR_CUDA;
        if (cudaFree(kv->joins) != cudaSuccess) r = AR_ERR_CUDA;
        return r;
    });
    k->magic = 0;
    delete k;
    return rc;
}

int ar_rope_append(ar_kv k, const ar_batch_t* b, const void* const* q, const void* const* kn, const void* const* vn,
                   void* const* q_out, int q_heads, size_t q_stride, size_t kv_stride, size_t q_out_stride,
                   const float* cos_sin, size_t max_positions, int rot_dim, int interleaved, ar_stream_t stream)
{
    KvCache* kv = get(k);
    if (!kv) return AR_ERR_INVALID;
    Handle& h = *kv->h;
    const RopeCall c{q, kn, vn, q_out, q_heads, q_stride, kv_stride, q_out_stride, cos_sin, max_positions, rot_dim,
                     interleaved};
    if (int rc = check_rope(h.n, kv->d, b, c)) return rc;
    const auto apart = [&](const void* const* rows, int heads, size_t stride) {
        return check_apart(h.n, kv->d, kv->k, kv->v, rows, (size_t)kv->d.head_dim * heads, stride, b->tokens);
    };
    if (int rc = apart(kn, kv->d.kv_heads, kv_stride)) return rc;
    if (int rc = apart(vn, kv->d.kv_heads, kv_stride)) return rc;
    if (q) {
        if (int rc = apart(q, q_heads, q_stride)) return rc;
        if (int rc = apart(q_out, q_heads, q_out_stride)) return rc;
    }
    const size_t row = (size_t)kv->d.head_dim * ((size_t)(q ? q_heads : 0) + 2u * (size_t)kv->d.kv_heads);
    int rc = AR_OK;
    h.timing.op = AR_OP_ROPE_APPEND;
    if (b->tokens) rc = on_device(h, [&] { return launch_rope_append(*kv, *b, c, (cudaStream_t)stream); });
    if (rc != AR_OK) return rc;
    const uint64_t moved = 2ull * h.n * b->tokens * row;
    note(h, AR_OP_ROPE_APPEND, b->tokens * row, moved, moved, (cudaStream_t)stream);
    return AR_OK;
}

int ar_paged_attention(ar_kv k, const ar_batch_t* b, const void* const* q, void* const* out, int q_heads,
                       size_t q_stride, size_t out_stride, float scale, int window, ar_stream_t stream)
{
    KvCache* kv = get(k);
    if (!kv) return AR_ERR_INVALID;
    Handle& h = *kv->h;
    const AttnCall c{q, out, q_heads, q_stride, out_stride, scale};
    if (int rc = check_attention(h.n, kv->d, b, c, window)) return rc;
    const size_t row = (size_t)kv->d.head_dim * (size_t)q_heads;
    if (int rc = check_apart(h.n, kv->d, kv->k, kv->v, out, row, out_stride, b->tokens)) return rc;
    int rc = AR_OK;
    h.timing.op = AR_OP_PAGED_ATTENTION;
    // The decode kernel reads a sequence's keys again for every row tile, the chunk kernel computes
    // 256 rows whatever there is.  Measured on GB300 (n = 4 bf16, 2 kv heads, us, decode / chunk) by
    // passes over the keys (query heads a kv head x new tokens), 64 sequences of 2000 keys:
    //   heads of 128: 1 (16 x 1) 95 / 118, 2 (8 x 4) 171 / 118;
    //   heads of 64:  1 (16 x 1) 57 / 96, 2 (8 x 4) 97 / 96, 3 (9 x 3) 135 / 96, 4 (8 x 8) 176 / 96,
    // and 16 sequences of 6000 keys: heads of 128: 1 73 / 87, 2 124 / 88; heads of 64: 2 65 / 69, 3 96 / 70.
    // (One sequence of 4000 keys is faster in the decode kernel up to 4 passes: 23.3 / 23.4, 16.4 / 21.)
    const bool few = decode_tiles(q_heads / kv->d.kv_heads, b->max_new).passes <= (kv->d.head_dim == 64 ? 2u : 1u);
    if (b->tokens)
        rc = on_device(h, [&] {
            return few ? launch_attention_decode(*kv, *b, c, window, (cudaStream_t)stream)
                       : launch_attention_chunk(*kv, *b, c, window, (cudaStream_t)stream);
        });
    if (rc != AR_OK) return rc;
    const uint64_t moved = 2ull * h.n * b->tokens * row;
    note(h, AR_OP_PAGED_ATTENTION, b->tokens * row, moved, moved, (cudaStream_t)stream);
    if (b->tokens && !few) h.last.launches = 2;
    return AR_OK;
}

}  // extern "C"
