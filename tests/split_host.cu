// Host program of test_attention_split_host.py: the units that the attention's
// split (csrc/paged.cuh) counts for sequences given as "new kv tm window" lines,
// with the decode kernel's key tiles (64, weight 1) and the chunk kernel's (128, 3).
#include <cstdio>

#include "paged.cuh"

int main()
{
    using namespace argb;
    int nq, len, tm, window;
    while (std::scanf("%d %d %d %d", &nq, &len, &tm, &window) == 4) {
        const Seq q{0, nq, len, len - nq};
        std::printf("%llu %llu\n", units_of_sequence<Split<64, 1, 4>>(q, tm, window),
                    units_of_sequence<Split<128, 3, 5>>(q, tm, window));
    }
    return 0;
}
