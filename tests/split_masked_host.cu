// Host program of test_attention_split_masked_host.py: the units that the scored attention's
// split (csrc/paged.cuh) counts for sequences given as "new kv tm window prefix documents" lines,
// documents: the first key of each new token's document, or 0 for none; with the decode kernel's key tiles
// (64, weight 1) and the chunk kernels' (128, 3 and 4).
#include <cstdio>
#include <vector>

#include "paged.cuh"

int main()
{
    using namespace argb;
    int nq, len, tm, window, prefix, documents;
    while (std::scanf("%d %d %d %d %d %d", &nq, &len, &tm, &window, &prefix, &documents) == 6) {
        std::vector<int32_t> first((size_t)(documents ? nq : 0));
        for (int32_t& x : first)
            if (std::scanf("%d", &x) != 1) return 1;
        MaskedBatchArgs b{};
        b.window = window;
        b.first = documents ? first.data() : nullptr;
        MaskedSeq q{};
        q.nq = nq;
        q.len = len;
        q.c0 = len - nq;
        q.prefix = prefix < len ? prefix : len;
        std::printf("%llu %llu %llu\n", units_in<Split<64, 1, 4>>(b, q, tm), units_in<Split<128, 3, 8>>(b, q, tm),
                    units_in<Split<128, 4, 12>>(b, q, tm));
    }
    return 0;
}
