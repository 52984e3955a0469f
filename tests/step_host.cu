// Host program of test_kv_step_reads_host.py: the table entry that kv_step_kernel reads for
// sequences given as "kv_len new_len done table_stride page_shift" lines before it knows whether the
// step can be served (-1: none), and whether it refuses the lengths.
#include <cstdio>

#include "kv_step.cuh"

int main()
{
    using namespace argb;
    int old, added, over, shift;
    size_t stride;
    while (std::scanf("%d %d %d %zu %d", &old, &added, &over, &stride, &shift) == 5) {
        const One o = one_of(old, added, over != 0, longest_row(stride, shift), shift);
        std::printf("%d %d\n", entry_of_one(o, shift), (int)(o.x.flags & kBad));
    }
    return 0;
}
