// Host-side internals of the calls around the all-reduce in a tensor-parallel
// layer (block norm, rotation and append, paged attention).  Not part of the
// C-ABI (that is include/ar.h).
#pragma once

#include <cuda.h>

#include "internal.h"

namespace argb {

constexpr int kAttnTileRows = 128;   // query rows of one tensor-core tile of the chunk kernel
constexpr int kMaxGroup = 64;        // query heads per kv head
constexpr float kLog2e = 1.4426950408889634f;   // the kernels' exponentials are powers of two

// The registered caches of a handle's ranks (ar_kv).
struct KvCache {
    Handle* h = nullptr;
    ar_kv_desc_t d{};
    int box_tokens = 0;              // tokens of one tensor copy: min(page_size, 64)
    void* encode = nullptr;          // the driver's cuTensorMapEncodeTiled
    void* k[kMaxRanks] = {};
    void* v[kMaxRanks] = {};
    CUtensorMap* maps = nullptr;     // device: n maps of K, then n of V
    float* partial = nullptr;        // device: partial results of rows split over CTAs
    unsigned* arrived = nullptr;     // device: decode kernel's partials arrived, by the CTA of the first part
    void* joins = nullptr;           // device: the chunk kernel's rows to join, by the CTA of the first part
};

// A call's batch and cache geometry, passed by value to the kernels.
struct BatchArgs {
    const int32_t* q_start;
    const int32_t* kv_len;
    const int32_t* table;
    size_t table_stride;
    int tokens, seqs;
    int page_shift;                  // log2(page_size)
    int pages;
    int window;                      // 0: none
    int absent;                      // rank whose keys never arrive at the attention kernels (-1: none)
};

inline BatchArgs batch_args(const KvCache& kv, const ar_batch_t& b, int window)
{
    // positions lie within 2^30 of 0 on both sides: a window of 2^30 is none, and differences fit 32 bits
    if (window > 1 << 30) window = 1 << 30;
    int shift = 4;
    while ((1 << shift) < kv.d.page_size) ++shift;
    return BatchArgs{b.q_start, b.kv_len, b.page_table, b.table_stride, (int)b.tokens, b.seqs, shift,
                     (int)kv.d.pages, window, kv.h->persist_absent};
}

// What the attention kernels take beside the batch.
struct AttnCall {
    const void* const* q;
    void* const* out;
    int q_heads;
    size_t q_stride, out_stride;     // elements
    float scale;
};

// A tensor map over 16-bit elements of the cache's type with the 128-byte
// swizzle; strides in bytes, of the second dimension on.
int encode_map(const KvCache& kv, CUtensorMap* map, int dims, const void* base, const size_t* size,
               const size_t* strides, const unsigned* box);

Handle* handle_of(ar_handle h);      // nullptr if it is not a handle

constexpr size_t kMaxNormHidden = 65536;   // 16 CTAs x 256 threads x 4 vectors of fp32
int launch_block_norm_f32(Handle& h, const void* const* in, const ar_block_norm_t& p, void* const* out,
                          void* residual_out, size_t tokens, size_t hidden, cudaStream_t s);
int launch_block_norm_bf16(Handle& h, const void* const* in, const ar_block_norm_t& p, void* const* out,
                           void* residual_out, size_t tokens, size_t hidden, cudaStream_t s);
int launch_block_norm_f16(Handle& h, const void* const* in, const ar_block_norm_t& p, void* const* out,
                          void* residual_out, size_t tokens, size_t hidden, cudaStream_t s);

struct RopeCall {
    const void* const* q;            // nullptr: none
    const void* const* k;
    const void* const* v;
    void* const* q_out;
    int q_heads;
    size_t q_stride, kv_stride, q_out_stride;
    const float* cos_sin;
    size_t max_positions;
    int rot_dim, interleaved;
};
int launch_rope_append(KvCache& kv, const ar_batch_t& b, const RopeCall& c, cudaStream_t s);

// The decode kernel's row tiles: whole tokens of up to 16 query heads of a kv head, 8
// rows if all rows of a sequence fit, else 16.
struct DecodeTiles {
    int rows;                        // 8 or 16
    int heads, head_groups;          // query heads of a tile, tiles that a kv head's take
    int tokens;                      // new tokens of a tile
    size_t passes;                   // how often the keys of a sequence with max_new new tokens are read
};

inline DecodeTiles decode_tiles(int group, int max_new)
{
    DecodeTiles t;
    t.rows = (size_t)max_new * (size_t)group <= 8 ? 8 : 16;
    t.heads = group < t.rows ? group : t.rows;
    t.head_groups = (group + t.heads - 1) / t.heads;
    t.tokens = t.rows / t.heads;
    t.passes = ((size_t)max_new + t.tokens - 1) / t.tokens * t.head_groups;
    return t;
}

size_t attention_decode_partial_floats(const Handle& h, int head_dim);
size_t attention_decode_counters(const Handle& h);
size_t attention_chunk_partial_floats(const Handle& h, int head_dim);
size_t attention_chunk_join_bytes(const Handle& h);
int launch_attention_decode(KvCache& kv, const ar_batch_t& b, const AttnCall& c, int window, cudaStream_t s);
int launch_attention_chunk(KvCache& kv, const ar_batch_t& b, const AttnCall& c, int window, cudaStream_t s);

}  // namespace argb
