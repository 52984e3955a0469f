// ar_allreduce_block_norm's kernels for fp32 payloads.
#include "block_norm.cuh"

namespace argb {

int launch_block_norm_f32(Handle& h, const void* const* in, const ar_block_norm_t& p, void* const* out,
                          void* residual_out, size_t tokens, size_t hidden, cudaStream_t s)
{
    return launch_block_norm_as<AR_F32>(h, in, p, out, residual_out, tokens, hidden, s);
}

}  // namespace argb
