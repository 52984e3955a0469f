// Rotation of the new tokens' queries and keys by their positions and append
// of keys and values to the ranks' paged caches, one launch for all ranks.
//
// Per pair (x1, x2) of a head and angle a = position * frequency, whose cosine
// c and sine s come from the caller's table: (x1 c - x2 s, x2 c + x1 s), in
// fp32, rounded once.  The call only moves bytes (each q, k, v element read
// and written once), so what bounds it is HBM for a prefill and the chain
// launch -> sequence -> page -> store for a decode step.
//
// Layout: a CTA takes one or more tokens of one rank; its threads take units
// of 16 elements (two 16-byte vectors that hold 8 whole pairs), so every
// access is 16 bytes and no pair crosses threads.  The data is loaded before
// the token's page is looked up: the two chains overlap.
#include "paged.cuh"

namespace argb {
namespace {

constexpr int kTh = 128;

struct RopePtrs {
    const void* q[kMaxRanks];
    const void* k[kMaxRanks];
    const void* v[kMaxRanks];
    void* q_out[kMaxRanks];
    void* kc[kMaxRanks];
    void* vc[kMaxRanks];
};

struct RopeArgs {
    int q_heads, kv_heads, dim;
    size_t q_stride, kv_stride, q_out_stride;
    size_t page_stride, head_stride, token_stride;
    const float* cos_sin;
    long long max_positions;
    int rot, interleaved;
};

// The sequence of token t: the last s with q_start[s] <= t.  A warp looks at
// 32 places of the range at once.
__device__ __forceinline__ int seq_of(const BatchArgs& b, int t, int lane)
{
    int lo = 0, hi = b.seqs;   // q_start[lo] <= t, answer in [lo, hi)
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) / 32;
        const int at = lo + lane * step;
        const bool below = at < hi && b.q_start[at] <= t;
        const int k = 31 - __clz(__ballot_sync(0xffffffffu, below) | 1u);
        const int nlo = lo + k * step;
        hi = min(hi, nlo + step);
        lo = nlo;
    }
    return lo;
}

template <int DT>
__global__ void __launch_bounds__(kTh)
rope_append_kernel(const __grid_constant__ RopePtrs p, const __grid_constant__ RopeArgs a, const BatchArgs b,
                   int units, int splits, DevStatus* st)
{
    using T = typename Payload<DT>::scalar_t;
    __shared__ long long sh_pos, sh_dst;   // position (-1: leave out), first element of the token's slot
    pdl_acquire();
    const int rank = blockIdx.z;
    const int t = blockIdx.x;
    const int half = a.dim / 16;                       // units of a head
    const int unit = blockIdx.y * kTh + threadIdx.x;
    const bool active = unit < units;
    const int head = active ? unit / half : 0, u = active ? unit % half : 0;
    const int hq = head, hk = head - a.q_heads, hv = hk - a.kv_heads;
    // the two vectors of this unit
    const bool is_v = hv >= 0;
    const int R = is_v ? 0 : a.rot;
    int e0 = 16 * u, e1 = e0 + 8;
    if (!a.interleaved && 16 * u < R) {
        e0 = 8 * u;
        e1 = e0 + R / 2;
    }
    const T* src = nullptr;
    uint4 x0 = make_uint4(0, 0, 0, 0), x1 = x0;
    if (active) {
        if (is_v)
            src = static_cast<const T*>(p.v[rank]) + (size_t)t * a.kv_stride + (size_t)hv * a.dim;
        else if (hk >= 0)
            src = static_cast<const T*>(p.k[rank]) + (size_t)t * a.kv_stride + (size_t)hk * a.dim;
        else
            src = static_cast<const T*>(p.q[rank]) + (size_t)t * a.q_stride + (size_t)hq * a.dim;
        x0 = ld16(src + e0);
        x1 = ld16(src + e1);
    }
    if (threadIdx.x < 32) {
        const int lane = threadIdx.x;
        const int s = seq_of(b, t, lane);
        if (lane == 0) {
            const Seq q = load_seq(b, s, st);
            long long pos = (long long)q.c0 + (t - q.q0), dst = -1;
            if (q.nq == 0 || t < q.q0 || t >= q.q0 + q.nq || pos < 0 || pos >= q.len ||
                (a.rot > 0 && pos >= a.max_positions)) {
                report_index(st);
                pos = -1;
            } else {
                const int page = b.table[(size_t)s * b.table_stride + (size_t)(pos >> b.page_shift)];
                if (page < 0 || page >= b.pages)
                    report_index(st);
                else
                    dst = (long long)page * (long long)a.page_stride +
                          (pos & ((1 << b.page_shift) - 1)) * (long long)a.token_stride;
            }
            sh_pos = pos;
            sh_dst = dst;
        }
    }
    __syncthreads();
    const long long pos = sh_pos, dst = sh_dst;
    pdl_release();
    if (!active || pos < 0 || dst < 0) return;
    if (16 * u < R) {
        const float* row = a.cos_sin + (size_t)pos * a.rot + 8 * u;
        float c[8], s[8], f[16], y[16];
#pragma unroll
        for (int k = 0; k < 8; k += 4) {
            *reinterpret_cast<float4*>(c + k) = __ldg(reinterpret_cast<const float4*>(row + k));
            *reinterpret_cast<float4*>(s + k) = __ldg(reinterpret_cast<const float4*>(row + a.rot / 2 + k));
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            Payload<DT>::widen(word(x0, j), f + 2 * j);
            Payload<DT>::widen(word(x1, j), f + 8 + 2 * j);
        }
        if (a.interleaved) {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                y[2 * k] = f[2 * k] * c[k] - f[2 * k + 1] * s[k];
                y[2 * k + 1] = f[2 * k + 1] * c[k] + f[2 * k] * s[k];
            }
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                y[k] = f[k] * c[k] - f[8 + k] * s[k];
                y[8 + k] = f[8 + k] * c[k] + f[k] * s[k];
            }
        }
        x0 = round_vec<DT>(y);
        x1 = round_vec<DT>(y + 8);
    }
    // the next call reads all of this: the stores keep the write-back policy
    if (hk < 0) {
        T* o = static_cast<T*>(p.q_out[rank]) + (size_t)t * a.q_out_stride + (size_t)hq * a.dim;
        st16_next(o + e0, x0);
        st16_next(o + e1, x1);
    } else {
        T* o = static_cast<T*>(is_v ? p.vc[rank] : p.kc[rank]) + dst + (size_t)(is_v ? hv : hk) * a.head_stride;
        st16_next(o + e0, x0);
        st16_next(o + e1, x1);
    }
}

}  // namespace

int launch_rope_append(KvCache& kv, const ar_batch_t& b, const RopeCall& c, cudaStream_t s)
{
    Handle& h = *kv.h;
    RopePtrs p{};
    for (int r = 0; r < h.n; ++r) {
        p.q[r] = c.q ? c.q[r] : nullptr;
        p.q_out[r] = c.q ? c.q_out[r] : nullptr;
        p.k[r] = c.k[r];
        p.v[r] = c.v[r];
        p.kc[r] = kv.k[r];
        p.vc[r] = kv.v[r];
    }
    const int qh = c.q ? c.q_heads : 0;
    RopeArgs a{qh, kv.d.kv_heads, kv.d.head_dim, c.q_stride, c.kv_stride, c.q_out_stride, kv.d.page_stride,
               kv.d.head_stride, kv.d.token_stride, c.cos_sin, (long long)c.max_positions, c.rot_dim, c.interleaved};
    const int units = (qh + 2 * kv.d.kv_heads) * (kv.d.head_dim / 16);
    const int splits = (units + kTh - 1) / kTh;
    const uint64_t moved = (uint64_t)h.n * b.tokens * (uint64_t)(qh + 2 * kv.d.kv_heads) * kv.d.head_dim * 2u;
    auto run = [&](auto dtc) -> int {
        constexpr int DT = decltype(dtc)::value;
        rec_begin(h, s);
        const cudaError_t e = launch_kernel(h, rope_append_kernel<DT>, dim3((unsigned)b.tokens, (unsigned)splits,
                                            (unsigned)h.n), dim3(kTh), 0, s, p, a, batch_args(kv, b, 0), units, splits,
                                            h.status);
        rec_end(h, s, AR_K_ROPE_APPEND, 2 * moved);
        return e == cudaSuccess ? launch_status() : AR_ERR_CUDA;
    };
    return kv.d.dtype == AR_BF16 ? run(std::integral_constant<int, AR_BF16>{})
                                 : run(std::integral_constant<int, AR_F16>{});
}

}  // namespace argb
