// A sequence's part of a step (kv_step.cu), from its lengths.
#pragma once

#include <cstddef>
#include <cstdint>

namespace argb {

enum : uint32_t { kBad = 1, kSeveralTokens = 2, kSeveralPages = 4 };

struct Sums {
    uint32_t tokens, take, give;
    uint32_t flags;
};

// One sequence of the step.
struct One {
    int kept, added, old;        // tokens that stay, new ones, tokens before
    Sums x;
};

// Tokens that a table row (and 2^30) can hold.
__host__ __device__ __forceinline__ int longest_row(size_t table_stride, int page_shift)
{
    const size_t row = table_stride << page_shift;
    return row < (size_t)1 << 30 ? (int)row : 1 << 30;
}

__host__ __device__ __forceinline__ One one_of(int old, int added, bool over, int longest, int page_shift)
{
    One o{over ? 0 : old, added, old, Sums{0, 0, 0, 0}};
    if (o.old < 0 || o.added < 0 || o.old > longest || o.added > longest - o.kept) {
        o.x.flags = kBad;
        return o;
    }
    auto pages = [&](int len) { return (uint32_t)(len + (1 << page_shift) - 1) >> page_shift; };
    o.x.tokens = (uint32_t)o.added;
    o.x.give = over ? pages(o.old) : 0u;
    o.x.take = pages(o.kept + o.added) - pages(o.kept);
    o.x.flags = (o.added > 1 ? kSeveralTokens : 0u) | (o.x.take > 1 ? kSeveralPages : 0u);
    return o;
}

// The entry of the sequence's table row that holds its single new token's page, where it
// has that page already; -1 where there is nothing to look up, and for lengths that are
// refused: they may point anywhere.
__host__ __device__ __forceinline__ int entry_of_one(const One& o, int page_shift)
{
    return o.added == 1 && o.x.take == 0 && !(o.x.flags & kBad) ? o.kept >> page_shift : -1;
}

}  // namespace argb
