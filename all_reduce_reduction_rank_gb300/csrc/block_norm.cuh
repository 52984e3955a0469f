// All-reduce fused with the norms around a block: sum over the ranks, norm of
// the block's output, gate, scaled residual, norm before the next block.
//
//   a = sum_r in_r;  b = a / sqrt(mean a^2 + eps) * w_post
//   r = alpha * residual + beta * gate * b;  y = r / sqrt(mean r^2 + eps) * w_pre
//
// The bytes bound it: n S + S (and the gate) read, n S + S written, a dozen
// flops per element.  Everything a thread loads (n ranks, residual, gate,
// weights) is issued before any of it is used, and a, r stay in fp32 registers
// between the two means, so each byte moves once and the row's two sums are
// the only waits.
//
// Measured on GB300 (n = 8, gate a row per token): 4096 x 8192 fp16, 1.275 GB: 200 us,
// 6.36 TB/s (95% of the copy rate); 61 x 8192 bf16 4.0 us; 1 x 4096 2.1 us, of which
// an empty launch in the same graph is most.
//
// One source per payload type includes this (they compile side by side).
//
// Layout: a cluster of CL CTAs per token row, each with a contiguous slice of
// it, VPT 16-byte vectors a thread.  Every warp sends its sum of squares into
// every CTA of the cluster (distributed shared memory, counted on the
// receiver's mbarrier), and every thread adds all of them in one order, so all
// CTAs get the same bits; one barrier for each of the two sums.
#pragma once

#include "cluster.cuh"
#include "layer.h"

namespace argb {
namespace {

struct NormArgs {
    const void* residual;
    const void* post;
    const void* gate;
    const void* pre;
    void* residual_out;
    size_t gate_stride;      // elements
    float alpha, beta, eps;
};

template <int DT>
__device__ __forceinline__ void widen_vec(const uint4& v, float* f)
{
#pragma unroll
    for (int j = 0; j < 4; ++j) Payload<DT>::widen(word(v, j), f + j * Payload<DT>::kPerWord);
}

template <int NR, int DT, int CL, int TH, int VPT>
__global__ void __launch_bounds__(TH, 512 / TH)
block_norm_kernel(const __grid_constant__ CPtrs<NR> in, const NormArgs a, const __grid_constant__ MPtrs<NR> out,
                  unsigned hidden, unsigned slice_vecs, int early_release, DevStatus* st)
{
    constexpr int VE = kVecElems<DT>;
    constexpr int W = TH / 32;
    constexpr int NP = CL * W;
    __shared__ float parts[2][NP];
    __shared__ __align__(8) uint64_t bars[2];
    if (threadIdx.x == 0) {
        cluster_bar_init(&bars[0], 4u * NP);
        cluster_bar_init(&bars[1], 4u * NP);
        cluster_bar_init_fence();
    }
    cluster_arrive();     // its wait, before the first sum is sent: every CTA has set up its barriers
    pdl_acquire();
    if (early_release) pdl_release();
    const unsigned c = cluster_ctarank();
    const size_t t = blockIdx.x / CL;
    const unsigned nvec = hidden / VE;
    const unsigned lo = c * slice_vecs, hi = min(lo + slice_vecs, nvec);
    const size_t row = t * nvec;
    const unsigned lane = threadIdx.x & 31, w = threadIdx.x >> 5;

    float f[VPT][VE];
    uint4 res[VPT], gate[VPT], post[VPT], pre[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const unsigned v = lo + threadIdx.x + i * TH;
        if (v < hi) {
            uint4 x[NR];
#pragma unroll
            for (int q = 0; q < NR; ++q) x[q] = ld16(static_cast<const uint4*>(in.p[q]) + row + v);
            res[i] = ld16(static_cast<const uint4*>(a.residual) + row + v);
            if (a.gate) gate[i] = ld16(static_cast<const uint4*>(a.gate) + t * (a.gate_stride / VE) + v);
            if (a.post) post[i] = ld16(static_cast<const uint4*>(a.post) + v);
            pre[i] = ld16(static_cast<const uint4*>(a.pre) + v);
#pragma unroll
            for (int k = 0; k < VE; ++k) f[i][k] = 0.0f;
#pragma unroll
            for (int q = 0; q < NR; ++q) accumulate<DT>(f[i], x[q]);
        }
    }
    // sum over the row of every thread's `ss`
    auto row_sum = [&](float ss, int k) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        if (lane < CL) st_async_cluster_f32(&parts[k][c * W + w], &bars[k], lane, ss);
        if (!cluster_bar_wait(&bars[k])) report_wait_timeout(st);
        float sum = 0.0f;
#pragma unroll
        for (int j = 0; j < NP; j += 32)
            if (j + (int)lane < NP) sum += parts[k][j + lane];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        return sum;
    };
    cluster_wait();
    float inv = 1.0f;
    if (a.post) {
        float ss = 0.0f;
#pragma unroll
        for (int i = 0; i < VPT; ++i)
            if (lo + threadIdx.x + i * TH < hi)
#pragma unroll
                for (int k = 0; k < VE; ++k) ss = fmaf(f[i][k], f[i][k], ss);
        inv = 1.0f / sqrtf(row_sum(ss, 0) / (float)hidden + a.eps);
    }
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const unsigned v = lo + threadIdx.x + i * TH;
        if (v < hi) {
            float x[VE];
            if (a.post) {
                widen_vec<DT>(post[i], x);
#pragma unroll
                for (int k = 0; k < VE; ++k) f[i][k] = f[i][k] * inv * x[k];
            }
            if (a.gate) {
                widen_vec<DT>(gate[i], x);
#pragma unroll
                for (int k = 0; k < VE; ++k) f[i][k] *= x[k];
            }
            widen_vec<DT>(res[i], x);
#pragma unroll
            for (int k = 0; k < VE; ++k) f[i][k] = fmaf(a.alpha, x[k], a.beta * f[i][k]);
            // the next block's epilogue reads it: the store keeps the write-back policy
            st16_next(static_cast<uint4*>(a.residual_out) + row + v, round_vec<DT>(f[i]));
#pragma unroll
            for (int k = 0; k < VE; ++k) ss = fmaf(f[i][k], f[i][k], ss);
        }
    }
    inv = 1.0f / sqrtf(row_sum(ss, 1) / (float)hidden + a.eps);
    if (!early_release) pdl_release();
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const unsigned v = lo + threadIdx.x + i * TH;
        if (v < hi) {
            float x[VE];
            widen_vec<DT>(pre[i], x);
#pragma unroll
            for (int k = 0; k < VE; ++k) f[i][k] = f[i][k] * inv * x[k];
            const uint4 y = round_vec<DT>(f[i]);
#pragma unroll
            for (int q = 0; q < NR; ++q) st16(static_cast<uint4*>(out.p[q]) + row + v, y);
        }
    }
}

template <int DT>
int launch_block_norm_as(Handle& h, const void* const* in, const ar_block_norm_t& p, void* const* out,
                         void* residual_out, size_t tokens, size_t hidden, cudaStream_t s)
{
    return dispatch_ranks(h.n, [&](auto nrc) -> int {
        constexpr int NR = decltype(nrc)::value;
        CPtrs<NR> ip;
        MPtrs<NR> op;
        for (int q = 0; q < NR; ++q) {
            ip.p[q] = in[q];
            op.p[q] = out[q];
        }
        NormArgs a{p.residual, p.post_weight, p.gate, p.pre_weight, residual_out,
                   p.gate ? p.gate_stride : 0, p.alpha, p.beta, p.eps};
        const uint64_t e = sizeof(typename Payload<DT>::scalar_t);
        const uint64_t S = (uint64_t)tokens * hidden * e, W = (uint64_t)hidden * e;
        const uint64_t extra = (p.gate ? (p.gate_stride ? S : W) : 0) + W * (p.post_weight ? 2 : 1);
        auto run = [&](auto clc, auto thc, auto vc) -> int {
            constexpr int CL = decltype(clc)::value, TH = decltype(thc)::value, VPT = decltype(vc)::value;
            auto kernel = block_norm_kernel<NR, DT, CL, TH, VPT>;
            static std::atomic<uint32_t> attr_done{0};
            if (CL > 8 && !once_per_device(attr_done, [&] {
                    return cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) ==
                           cudaSuccess;
                }))
                return AR_ERR_CUDA;
            const unsigned slice = (unsigned)((hidden / kVecElems<DT> + CL - 1) / CL);
            cudaLaunchAttribute attr[2];
            attr[0].id = cudaLaunchAttributeClusterDimension;
            attr[0].val.clusterDim.x = CL;
            attr[0].val.clusterDim.y = 1;
            attr[0].val.clusterDim.z = 1;
            attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
            attr[1].val.programmaticStreamSerializationAllowed = h.pdl ? 1 : 0;
            cudaLaunchConfig_t cfg{};
            cfg.gridDim = dim3((unsigned)(tokens * CL));
            cfg.blockDim = dim3(TH);
            cfg.stream = s;
            cfg.attrs = attr;
            cfg.numAttrs = 2;
            const int early = tokens * CL <= (size_t)h.sm_count ? 1 : 0;
            rec_begin(h, s);
            const cudaError_t err = cudaLaunchKernelEx(&cfg, kernel, ip, a, op, (unsigned)hidden, slice, early,
                                                       h.status);
            rec_end(h, s, AR_K_ALLREDUCE_BLOCK_NORM, 2ull * (NR + 1) * S + extra);
            return err == cudaSuccess ? launch_status() : AR_ERR_CUDA;
        };
        using C1 = std::integral_constant<int, 1>;
        using C2 = std::integral_constant<int, 2>;
        using C4 = std::integral_constant<int, 4>;
        using C8 = std::integral_constant<int, 8>;
        using C16 = std::integral_constant<int, 16>;
        using T128 = std::integral_constant<int, 128>;
        using T256 = std::integral_constant<int, 256>;
        // Clusters just wide enough for one vector a thread of 128, so that a row's
        // phases overlap another's on the same SM; up to 8 CTAs for rows too few to
        // fill the SMs; two vectors a thread on 4 CTAs instead of one on 8 once the
        // rows are many.  Swept on GB300 (n = 8 bf16, graph replay, every {1, 2, 4, 8,
        // 16} CTAs x {64 ... 512} threads x {1, 2, 4} vectors): the best or within 4%
        // of it at 1 x 4096 (2.1 us), 61 x 8192 (4.0), 128 x 4096 (3.9), 1000 x 512
        // (4.5), 2000 x 1864 (25.4), 2000 x 4096 (50.3), 2000 x 16384 (201);
        // 300 x 8192 (17.6; 16.5 with four vectors on 2 CTAs, which lose elsewhere).
        // 4096 x 8192: 201 us with two vectors on 4 CTAs, 207 with one on 8.
        const size_t nvec = hidden / kVecElems<DT>;
        if (nvec <= 1024 && tokens * 8 <= (size_t)h.sm_count) return run(C8{}, T128{}, C1{});
        if (nvec <= 128) return run(C1{}, T128{}, C1{});
        if (nvec <= 256) return run(C2{}, T128{}, C1{});
        if (nvec <= 512) return run(C4{}, T128{}, C1{});
        if (nvec <= 1024) return tokens < 1024 ? run(C8{}, T128{}, C1{}) : run(C4{}, T128{}, C2{});
        if (nvec <= 2048) return run(C8{}, T128{}, C2{});
        if (nvec <= 4096) return run(C16{}, T128{}, C2{});
        return run(C16{}, T256{}, C4{});
    });
}

}  // namespace
}  // namespace argb
