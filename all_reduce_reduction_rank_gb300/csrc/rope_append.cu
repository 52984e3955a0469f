// Rotation of the new tokens' queries and keys by their positions and append
// of keys and values to the ranks' paged caches, one launch for all ranks.
//
// Per pair (x1, x2) of a head and angle a = position * frequency, whose cosine
// c and sine s come from the caller's table: (x1 c - x2 s, x2 c + x1 s), in
// fp32, rounded once.  The call only moves bytes (each q, k, v element read
// and written once), so what bounds it is HBM for a prefill and the chain
// launch -> sequence -> page -> store for a decode step.
//
// Layout: a thread takes the same 16 elements (two 16-byte vectors that hold 8
// whole pairs) of HEADS heads of a token, so every access is 16 bytes and no pair
// crosses threads.  A CTA takes up to 4 tokens of one rank, a warp looking up
// each one's sequence, position and page; the data is loaded before that is
// waited for, so the two chains overlap.  HEADS is 4 for many tokens: a table row
// is loaded once for 4 heads (a thread a head spent half its time issuing, 282
// instructions for 64 bytes); 1, with a token a CTA, for few: the shorter chain.
// Measured on GB300 (us, 4 / 1): 8000 tokens on 4 ranks (198 MB) 34.0 / 43.8, 87%
// of the copy rate; 436 on 8 ranks 3.2 / 5.1; 61 on 8 ranks 3.1 / 2.7; 1 on 8
// ranks 2.5 / 2.05.
#include <algorithm>

#include "paged.cuh"

namespace argb {
namespace {

constexpr int kTh = 128;
constexpr int kMaxTokens = 4;    // tokens of a CTA, a warp each

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
    int unit_shift;          // log2 of the 16-element units of a head
    int groups, per_token;   // threads of a token: groups of heads x units
    int cta_tokens;
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

template <int DT, int HEADS>
__global__ void __launch_bounds__(kTh)
rope_append_kernel(const __grid_constant__ RopePtrs p, const __grid_constant__ RopeArgs a, const BatchArgs b,
                   DevStatus* st)
{
    using T = typename Payload<DT>::scalar_t;
    __shared__ long long sh_pos[kMaxTokens], sh_dst[kMaxTokens];   // position (-1: leave out), its slot's first element
    pdl_acquire();
    const int rank = blockIdx.z, t0 = blockIdx.x * a.cta_tokens;
    const int item = blockIdx.y * kTh + threadIdx.x;
    const int w = item / a.per_token, r = item - w * a.per_token, t = t0 + w;
    const bool active = w < a.cta_tokens && t < b.tokens;
    const int u = r & ((1 << a.unit_shift) - 1), first = r >> a.unit_shift;   // 16 elements of a head, first head
    const int heads = a.q_heads + 2 * a.kv_heads, turned = a.q_heads + a.kv_heads;
    // the two vectors: neighbours, or R/2 apart where they hold the two sides of the pairs
    const bool in_turn = 16 * u < a.rot;
    const int t_e0 = in_turn && !a.interleaved ? 8 * u : 16 * u;
    const int t_e1 = in_turn && !a.interleaved ? t_e0 + a.rot / 2 : t_e0 + 8;
    uint4 x0[HEADS], x1[HEADS];
    if (active) {
#pragma unroll
        for (int k = 0; k < HEADS; ++k) {
            const int h = first + k * a.groups;
            if (h >= heads) break;
            const T* src;
            if (h < a.q_heads)
                src = static_cast<const T*>(p.q[rank]) + (size_t)t * a.q_stride + (size_t)h * a.dim;
            else if (h < turned)
                src = static_cast<const T*>(p.k[rank]) + (size_t)t * a.kv_stride + (size_t)(h - a.q_heads) * a.dim;
            else
                src = static_cast<const T*>(p.v[rank]) + (size_t)t * a.kv_stride + (size_t)(h - turned) * a.dim;
            x0[k] = ld16(src + (h < turned ? t_e0 : 16 * u));
            x1[k] = ld16(src + (h < turned ? t_e1 : 16 * u + 8));
        }
    }
    const int warp = threadIdx.x / 32;
    if (warp < a.cta_tokens && t0 + warp < b.tokens) {
        const int lane = threadIdx.x & 31, mine = t0 + warp;
        const int s = seq_of(b, mine, lane);
        if (lane == 0) {
            const Seq q = load_seq(b, s, st);
            long long pos = (long long)q.c0 + (mine - q.q0), dst = -1;
            if (q.nq == 0 || mine < q.q0 || mine >= q.q0 + q.nq || pos < 0 || pos >= q.len ||
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
            sh_pos[warp] = pos;
            sh_dst[warp] = dst;
        }
    }
    __syncthreads();
    pdl_release();
    if (!active) return;
    const long long pos = sh_pos[w], dst = sh_dst[w];
    if (pos < 0 || dst < 0) return;
    float c[8], s[8];
    if (in_turn && first < turned) {
        const float* row = a.cos_sin + (size_t)pos * a.rot + 8 * u;
#pragma unroll
        for (int k = 0; k < 8; k += 4) {
            *reinterpret_cast<float4*>(c + k) = __ldg(reinterpret_cast<const float4*>(row + k));
            *reinterpret_cast<float4*>(s + k) = __ldg(reinterpret_cast<const float4*>(row + a.rot / 2 + k));
        }
    }
#pragma unroll
    for (int k = 0; k < HEADS; ++k) {
        const int h = first + k * a.groups;
        if (h >= heads) break;
        if (in_turn && h < turned) {
            float f[16], y[16];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                Payload<DT>::widen(word(x0[k], j), f + 2 * j);
                Payload<DT>::widen(word(x1[k], j), f + 8 + 2 * j);
            }
            if (a.interleaved) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    y[2 * j] = fmaf(f[2 * j], c[j], -(f[2 * j + 1] * s[j]));
                    y[2 * j + 1] = fmaf(f[2 * j + 1], c[j], f[2 * j] * s[j]);
                }
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    y[j] = fmaf(f[j], c[j], -(f[8 + j] * s[j]));
                    y[8 + j] = fmaf(f[8 + j], c[j], f[j] * s[j]);
                }
            }
            x0[k] = round_vec<DT>(y);
            x1[k] = round_vec<DT>(y + 8);
        }
        // the next call reads all of this: the stores keep the write-back policy
        T* o;
        if (h < a.q_heads)
            o = static_cast<T*>(p.q_out[rank]) + (size_t)t * a.q_out_stride + (size_t)h * a.dim;
        else if (h < turned)
            o = static_cast<T*>(p.kc[rank]) + dst + (size_t)(h - a.q_heads) * a.head_stride;
        else
            o = static_cast<T*>(p.vc[rank]) + dst + (size_t)(h - turned) * a.head_stride;
        st16_next(o + (h < turned ? t_e0 : 16 * u), x0[k]);
        st16_next(o + (h < turned ? t_e1 : 16 * u + 8), x1[k]);
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
    const int heads = qh + 2 * kv.d.kv_heads;
    RopeArgs a{};
    a.q_heads = qh;
    a.kv_heads = kv.d.kv_heads;
    a.dim = kv.d.head_dim;
    a.q_stride = c.q_stride;
    a.kv_stride = c.kv_stride;
    a.q_out_stride = c.q_out_stride;
    a.page_stride = kv.d.page_stride;
    a.head_stride = kv.d.head_stride;
    a.token_stride = kv.d.token_stride;
    a.cos_sin = c.cos_sin;
    a.max_positions = (long long)c.max_positions;
    a.rot = c.rot_dim;
    a.interleaved = c.interleaved;
    a.unit_shift = kv.d.head_dim == 128 ? 3 : 2;
    const uint64_t moved = (uint64_t)h.n * b.tokens * (uint64_t)(qh + 2 * kv.d.kv_heads) * kv.d.head_dim * 2u;
    auto run = [&](auto dtc, auto hc) -> int {
        constexpr int DT = decltype(dtc)::value, HEADS = decltype(hc)::value;
        a.groups = (heads + HEADS - 1) / HEADS;
        a.per_token = a.groups << a.unit_shift;
        a.cta_tokens = HEADS == 1 || a.per_token >= kTh ? 1 : std::min(kTh / a.per_token, kMaxTokens);
        const unsigned splits = (unsigned)((a.cta_tokens * a.per_token + kTh - 1) / kTh);
        rec_begin(h, s);
        const cudaError_t e = launch_kernel(
            h, rope_append_kernel<DT, HEADS>,
            dim3((unsigned)((b.tokens + a.cta_tokens - 1) / a.cta_tokens), splits, (unsigned)h.n), dim3(kTh), 0, s, p, a,
            batch_args(kv, b, 0), h.status);
        rec_end(h, s, AR_K_ROPE_APPEND, 2 * moved);
        return e == cudaSuccess ? launch_status() : AR_ERR_CUDA;
    };
    auto sized = [&](auto dtc) -> int {
        return b.tokens * (size_t)h.n > 1024 ? run(dtc, std::integral_constant<int, 4>{})
                                             : run(dtc, std::integral_constant<int, 1>{});
    };
    return kv.d.dtype == AR_BF16 ? sized(std::integral_constant<int, AR_BF16>{})
                                 : sized(std::integral_constant<int, AR_F16>{});
}

}  // namespace argb
