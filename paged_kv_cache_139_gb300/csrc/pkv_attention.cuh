// What the decode kernels over the 16-bit and the 8-bit cache share: their
// arguments, the partition partials and their log-sum-exp merge (inside the
// kernel and in a kernel of its own).
#pragma once

#include <cmath>

#include "pkv_host.cuh"

namespace pkv {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float warp_max(float x) {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) x = fmaxf(x, __shfl_xor_sync(kFull, x, o));
    return x;
}

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) x += __shfl_xor_sync(kFull, x, o);
    return x;
}

struct AttnArgs {
    void *out;                   // [S][H][D] T
    float *ws_m;                 // [S][H][MP]
    float *ws_l;                 // [S][H][MP]
    float *ws_o;                 // [S][H][MP][D]
    const void *q;               // [S][H][D]
    const void *k_cache;         // [NB][Hkv][B][D]
    const void *v_cache;
    const int32_t *tables;       // [S][max_blocks]
    const int32_t *ctx_lens;     // [S]
    DeviceStatus *st;
    WsHeader *hdr;               // work-ticket counters at the head of the workspace
    int num_seqs;
    int max_blocks;
    int max_ctx;
    int log2_block;
    int num_blocks;
    int num_heads;
    int num_kv_heads;
    int head_tiles;              // (H / Hkv) / G
    int partition;               // P
    int max_parts;               // MP
    float scale_log2;            // scale * log2(e)
    unsigned int *cnt;           // [S][H] partitions finished (fused merge); zero between calls
    int fused_merge;             // 1: the last partition of a (sequence, head tile) merges them all
    // the step's new tokens, written into the cache by the kernel (null: already written)
    const void *new_k;           // [S][Hkv][D]
    const void *new_v;
    const int64_t *slots;        // [S]
};

// Splits of up to this many partitions merge inside the attention kernel:
// the CTA that completes the last partition of a (sequence, query-head tile)
// -- found by an atomic counter -- merges them.  Longer splits go to
// partition_reduce_kernel.
#ifndef PKV_FUSED_MAX_PARTS
#define PKV_FUSED_MAX_PARTS 16
#endif
constexpr int kFusedMaxParts = PKV_FUSED_MAX_PARTS;
static_assert(kFusedMaxParts <= 32, "the in-kernel merge keeps one partition per lane");

// Log-sum-exp merge, by one warp, of the np partitions of query heads
// h0 .. h0 + heads - 1 of sequence s (np <= 32, one per lane):
// M = max m_p, L = sum l_p 2^(m_p - M), out = sum o_p 2^(m_p - M) / L.
// Lane L owns D/32 consecutive elements of a row.  The partials were written
// by other CTAs: they are read past L1.  A head's m, l and first 8 rows are
// loaded together, so a head costs one round trip per 8 partitions.
template <int D, typename T>
__device__ __forceinline__ void merge_partitions_warp(const AttnArgs &a, int s, int h0, int heads, int np, int lane) {
    constexpr int EPL = D / 32;
#pragma unroll 1
    for (int h = 0; h < heads; h++) {
        const size_t base = ((size_t)s * a.num_heads + h0 + h) * a.max_parts;
        const float mp = lane < np ? __ldcg(a.ws_m + base + lane) : -INFINITY;
        const float lp = lane < np ? __ldcg(a.ws_l + base + lane) : 0.f;
        float acc[EPL];
#pragma unroll
        for (int k = 0; k < EPL; k++) acc[k] = 0.f;
        float wp = 0.f;
#pragma unroll 1
        for (int p0 = 0; p0 < np; p0 += 8) {
            float ov[8][EPL];
#pragma unroll
            for (int j = 0; j < 8; j++) {
                const float *src = a.ws_o + (base + p0 + j) * D + lane * EPL;
                if (p0 + j < np) {
                    if constexpr (EPL == 4) {
                        const float4 v = __ldcg(reinterpret_cast<const float4 *>(src));
                        ov[j][0] = v.x; ov[j][1] = v.y; ov[j][2] = v.z; ov[j][3] = v.w;
                    } else {
                        const float2 v = __ldcg(reinterpret_cast<const float2 *>(src));
                        ov[j][0] = v.x; ov[j][1] = v.y;
                    }
                } else {
#pragma unroll
                    for (int k = 0; k < EPL; k++) ov[j][k] = 0.f;
                }
            }
            if (p0 == 0) {                       // uniform: the weights, while the first rows load
                const float M = warp_max(mp);
                wp = lane < np ? exp2f(mp - M) : 0.f;
            }
#pragma unroll
            for (int j = 0; j < 8; j++) {
                const float w = __shfl_sync(kFull, wp, (p0 + j) & 31);
#pragma unroll
                for (int k = 0; k < EPL; k++) acc[k] = fmaf(w, ov[j][k], acc[k]);
            }
        }
        const float L = warp_sum(lp * wp);
        T *dst = static_cast<T *>(a.out) + ((size_t)s * a.num_heads + h0 + h) * D + lane * EPL;
#pragma unroll
        for (int k = 0; k < EPL; k++) dst[k] = F16Traits<T>::from_f32(L > 0.f ? acc[k] / L : 0.f);
    }
}

// Merge the partitions of each (sequence, head) with more than one:
// M = max_p m_p, L = sum_p l_p 2^(m_p - M), out = sum_p o_p 2^(m_p - M) / L.
// One CTA per (head, sequence).  Thread t owns the 16-byte column t % CPR of
// the partial rows t / CPR, t / CPR + RG, ... of a chunk of RG * kReduceRows
// partitions: a chunk's rows are all requested at once, before the weights
// they need are known, so a split of up to one chunk (64 partitions at
// head_dim 128) costs about two round trips to L2.
constexpr int kReduceThreads = 256;
constexpr int kReduceRows = 8;                      // partial rows per thread per chunk

template <int D, typename T>
__global__ void __launch_bounds__(kReduceThreads) partition_reduce_kernel(const AttnArgs a) {
    constexpr int CPR = D / 4;                      // float4 columns per row
    constexpr int RG = kReduceThreads / CPR;        // row groups
    constexpr int CH = RG * kReduceRows;            // partitions per chunk
    static_assert(CH <= kReduceThreads, "one weight per thread and chunk");
    __shared__ float wsh[CH];
    __shared__ float red[2][kReduceThreads / 32];
    __shared__ float4 opart[RG][CPR];
    pdl_trigger();
    pdl_wait();
    const int h = blockIdx.x, s = blockIdx.y, tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
    int ctx = a.ctx_lens[s];
    ctx = ctx < 0 ? 0 : (ctx > a.max_ctx ? a.max_ctx : ctx);
    const int np = (ctx + a.partition - 1) / a.partition;
    if (np <= 1) return;                            // uniform over the CTA
    const size_t base = ((size_t)s * a.num_heads + h) * a.max_parts;
    const float *m = a.ws_m + base;
    const float *l = a.ws_l + base;
    const float4 *o = reinterpret_cast<const float4 *>(a.ws_o + base * D);
    const int c = tid % CPR, rg = tid / CPR;
    float4 ov[kReduceRows];
    auto load_chunk = [&](int p0) {
#pragma unroll
        for (int k = 0; k < kReduceRows; k++) {
            const int p = p0 + rg + RG * k;
            ov[k] = p < np ? __ldcg(o + (size_t)p * CPR + c) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
    };
    // the first chunk's rows and the first kReduceThreads (m, l) are requested together
    load_chunk(0);
    const float m0 = tid < np ? __ldcg(m + tid) : -INFINITY;
    const float l0 = tid < np ? __ldcg(l + tid) : 0.f;
    float mx = m0;
    for (int p = tid + kReduceThreads; p < np; p += kReduceThreads) mx = fmaxf(mx, __ldcg(m + p));
    mx = warp_max(mx);
    if (lane == 0) red[0][wid] = mx;
    __syncthreads();
    float M = red[0][0];
#pragma unroll
    for (int w = 1; w < kReduceThreads / 32; w++) M = fmaxf(M, red[0][w]);
    const float w0 = tid < np ? exp2f(m0 - M) : 0.f;
    float lp = l0 * w0;
    for (int p = tid + kReduceThreads; p < np; p += kReduceThreads)
        lp = fmaf(__ldcg(l + p), exp2f(__ldcg(m + p) - M), lp);
    lp = warp_sum(lp);
    if (lane == 0) red[1][wid] = lp;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int p0 = 0; p0 < np; p0 += CH) {
        if (p0 > 0) load_chunk(p0);
        if (tid < CH) wsh[tid] = p0 == 0 ? w0 : (p0 + tid < np ? exp2f(__ldcg(m + p0 + tid) - M) : 0.f);
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kReduceRows; k++) {
            const float w = wsh[rg + RG * k];
            acc.x = fmaf(w, ov[k].x, acc.x);
            acc.y = fmaf(w, ov[k].y, acc.y);
            acc.z = fmaf(w, ov[k].z, acc.z);
            acc.w = fmaf(w, ov[k].w, acc.w);
        }
        __syncthreads();
    }
    opart[rg][c] = acc;
    __syncthreads();
    if (rg == 0) {
        float L = 0.f;
#pragma unroll
        for (int w = 0; w < kReduceThreads / 32; w++) L += red[1][w];
#pragma unroll
        for (int g = 1; g < RG; g++) {
            const float4 x = opart[g][c];
            acc.x += x.x; acc.y += x.y; acc.z += x.z; acc.w += x.w;
        }
        T *dst = static_cast<T *>(a.out) + ((size_t)s * a.num_heads + h) * D + c * 4;
        dst[0] = F16Traits<T>::from_f32(L > 0.f ? acc.x / L : 0.f);
        dst[1] = F16Traits<T>::from_f32(L > 0.f ? acc.y / L : 0.f);
        dst[2] = F16Traits<T>::from_f32(L > 0.f ? acc.z / L : 0.f);
        dst[3] = F16Traits<T>::from_f32(L > 0.f ? acc.w / L : 0.f);
    }
}

template <typename T> cudaError_t launch_reduce(int D, const AttnArgs &a, dim3 grid, cudaStream_t st) {
    if (D == 64) return launch(partition_reduce_kernel<64, T>, grid, dim3(kReduceThreads), 0, st, a);
    return launch(partition_reduce_kernel<128, T>, grid, dim3(kReduceThreads), 0, st, a);
}

inline int parts_for(int max_ctx, int P) { return max_ctx > 0 ? (int)(((long long)max_ctx + P - 1) / P) : 1; }

// P as the kernels take it: they round lengths up to it in 31 bits, so one that is
// longer than every context becomes the least multiple of `step` that holds them.
inline int kernel_partition(int P, int max_ctx, int step) {
    const long long all = ((long long)max_ctx + step - 1) / step * step;
    const long long most = all < step ? step : all > (1 << 30) ? 1 << 30 : all;
    return P < most ? P : (int)most;
}

inline size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

}  // namespace
}  // namespace pkv
