// Paged decode attention over the 8-bit cache, and the prompt phase over it.
//
// What it computes: for sequence s, query head h and its kv head g,
//     out = sum_t softmax_t(scale * q . k_t) v_t,
//     k_t = e4m3 code * scales[b][g][0],  v_t = e4m3 code * scales[b][g][1],
// token t in block b = block_tables[s][t / B] at offset t % B.
//
// Decode is bound by the bytes of the cache, half those of a 16-bit one, so
// there are twice the tokens per byte to compute on: at 7 TB/s an SM has to
// take in about 24 codes a clock.  So the products run on the tensor cores
// for every group of query heads, one included, and what each code costs is
// kept down to its share of a conversion:
//   * S^T = K Q^T and O^T = V^T P^T: the cache's codes are the 16-row operand
//     of both products and the query heads of a kv head (up to 8) the 8
//     columns.  A code converts exactly to fp16, two at a time, straight into
//     the fragment: the products' inner index and rows may be numbered at
//     will, so a lane takes sixteen consecutive codes of a token with one load
//     and K needs no transposition; for V two tokens' bytes are interleaved
//     (one byte permute per two fragment registers).  fp16 queries enter as
//     they are, bf16 ones scaled by a power of two per head into fp16's range.
//   * Up to four heads leave four columns idle: those repeat the heads and
//     carry what fp16 loses of the probabilities, so that P V has 22 bits of P
//     at no extra product.  More heads take a second product for it.
//   * The key scale multiplies the finished score, the value scale the
//     probability, relative to the largest value scale so far: a probability
//     enters the product as 2^(x - m) * (scale / largest) * 2^15, which fits
//     fp16 with 24 bits to spare below it.  Where an item's value scales
//     spread over more than 2^10, that could lose the blocks of small scales;
//     there the reference is the running maximum of x + log2(scale) instead.
//   * K and V tiles come by tiled TMA, swizzled; tokens are numbered within
//     groups of eight so that the wide loads of both are free of bank
//     conflicts (see perm_token).
// A CTA is four pipelines of a producer and a consumer warp, one consumer to
// each of the SM's schedulers, two CTAs to an SM; each pipeline is persistent
// over (sequence, partition, head tile) items that it claims by tickets.  The
// partitions of a split context are merged by a second kernel: merging in this
// one (a fence and an atomic per item) cost more than its launch.
//
// Measured: 256 x uniform[1, 4096] tokens of 32 heads x 128 (4.5 GB) 632 us, 7.1
// TB/s; 64 sequences of 40 heads, 288 MB, 52 us; 8 x 32,768 tokens of 8 kv heads,
// 538 MB, 90 us with 6 us of merging.  More than eight query heads per kv head take a
// head tile each, which reads and converts its tiles again: 537 MB in 94 us at 32/4
// heads, in 167 us at 32/2.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <climits>
#include <cstring>
#include <type_traits>

#include "pkv_attention.cuh"
#include "pkv_fp8.cuh"
#include "pkv_host.cuh"
#include "pkv_tmap.h"

namespace pkv {
namespace {

// Tuning knob (compile-time): ring slots of a pipeline.
#ifndef PKV_FP8_SLOTS
#define PKV_FP8_SLOTS 3
#endif
constexpr int kPipes = 4;                   // pipelines of a CTA
constexpr int kCtasPerSm = 2;
constexpr int kStageBytes = 4096;           // a ring stage's K, and its V: 32 tokens at head_dim 128, 64 at 64
constexpr int kMaxTokens = kStageBytes / 64;
constexpr int kMinBlock = 4;
constexpr int kStageBlocks = kMaxTokens / kMinBlock;
constexpr int kTileHeads = 8;               // query heads per item at most: the products' columns
constexpr int kLaunchSeqs = 512;            // sequences per launch (their lengths sit in shared memory)
constexpr int kMaxSpread = 10;              // log2 of the largest over the least value scale, see above
constexpr int kPExp = 15;                   // probabilities enter the product times 2^15 (fp16 reaches 2^16)

// The workspace: two ticket headers (decode; the prompt phase at 128), then
// what a call needs.  Every call leaves the headers ready: calls of any sizes,
// captured or not, may follow one another on a workspace.
constexpr size_t kPrefillHeader = 128;
constexpr size_t kBodyOff = kWsHeaderBytes;

struct F8Args {
    AttnArgs a;
    const float2 *scales;        // [NB][scale_heads]
    int scale_heads;
    int tile;                    // query heads per item (the last tile of a kv head may hold fewer)
};

struct F8Meta {
    int s, h0, rows, part, nparts;   // the item: query heads h0 .. h0 + rows - 1
    int nvalid;                      // tokens of the stage
    int flags;
    int range;                       // value scales of the item's blocks up to here: see scale_range
};

// A pipeline's shared memory, and the CTA's.
struct F8Layout {
    static constexpr int R = PKV_FP8_SLOTS;
    static constexpr uint32_t ring = 0;                                             // [R][2][kStageBytes]
    static constexpr uint32_t q = ring + R * 2 * kStageBytes;                       // [8][<= 128] 16-bit
    static constexpr uint32_t sc = q + kTileHeads * 128 * 2;                        // [R][kStageBlocks] float2
    static constexpr uint32_t bars = sc + R * kStageBlocks * 8;
    static constexpr uint32_t meta = bars + 2 * R * 8;
    static constexpr uint32_t bytes = meta + R * sizeof(F8Meta);
    // the 128-byte swizzle repeats every 1024 bytes: rings start on such a boundary, in front of the rest
    static constexpr uint32_t rings = 0;
    static constexpr uint32_t rest = kPipes * q;
    static constexpr uint32_t rest_bytes = bytes - q;
    static constexpr uint32_t misc = rest + kPipes * rest_bytes;
    static constexpr uint32_t seqs = misc + 64 * 4;
    static size_t total(int S) { return seqs + (size_t)(2 * S + 1) * sizeof(int); }
    static_assert(q % 1024 == 0 && rest_bytes % 16 == 0, "swizzled rings, 16-byte copies");
};

enum : int { kFirst = 1, kLast = 2, kStop = 4 };

// Row j of a group of eight is its token perm_token(j).  The numbers make the
// quarter-warps of the wide loads hit distinct banks: of K, rows 2i and 2i + 1
// (four chunks each); of V, the four even or the four odd rows (two chunks
// each), under the swizzle of 128- or 64-byte rows.
template <int D> __device__ __forceinline__ int perm_token(int j) {
    if (D >= 128) return j ^ ((j & 1) << 2);                              // 0 5 2 7 4 1 6 3
    const int even = ((j & 2) << 1) | (j >> 2);                           // 0 4 1 5 of columns 0 2 4 6
    return (j & 1) ? even ^ 3 : even;                                     // 0 3 4 7 1 2 5 6
}

// Byte offset of 16-byte chunk `chunk` of token row `row` in a stage.
template <int D> __device__ __forceinline__ int chunk_at(int row, int chunk) {
    if (D >= 128) return row * 128 + ((chunk ^ (row & 7)) << 4);
    return row * 64 + ((chunk ^ ((row >> 1) & 3)) << 4);
}

// The lane's two columns (2c and 2c + 1, c = lane % 4) of an item.  o is the
// value sum relative to 2^(r - 15): r = m + (log2 of the largest value scale so
// far), or above the largest x + log2(scale) where scales spread far.
template <int D> struct F8State {
    float o[D / 16][4];    // d = (D / 8) (lane / 4) + 2 i: [0], [1]; + 1: [2], [3]
    float m[2], l[2];      // running max (log2 domain) and this lane's share of the sum of exponentials
    float r[2];
};

template <int D> __device__ __forceinline__ void f8_reset(F8State<D> &st) {
#pragma unroll
    for (int j = 0; j < D / 16; j++)
#pragma unroll
        for (int e = 0; e < 4; e++) st.o[j][e] = 0.f;
#pragma unroll
    for (int e = 0; e < 2; e++) {
        st.m[e] = st.r[e] = -INFINITY;
        st.l[e] = 0.f;
    }
}

// 2^x: the hardware's approximation (relative error 2^-22), subnormal results flushed.
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// The 8x8 matrix of 16-bit elements whose row lane / 4, columns 2c and 2c + 1
// each lane holds, transposed.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// The largest exponent of the value scales seen (the scale is at most 2^top),
// and whether they spread over more than 2^kMaxSpread; negative and zero
// scales count as far below.
__device__ __forceinline__ int scale_range(int top, int low) {
    return top * 2 + (top - low > kMaxSpread ? 1 : 0);
}
// e with 2^(e - 1) < v <= 2^e.
__device__ __forceinline__ int exponent_above(float v) {
    if (!(v > 0.f)) return -1000;
    const unsigned b = __float_as_uint(v);
    return (int)(b >> 23) - 127 + ((b & 0x7fffffu) ? 1 : 0);
}

// Query head lane / 4 (of an item of `rows`; the upper four columns repeat the
// lower ones unless WIDE) as B fragments.  k-step ks of lane column c covers
// d = (ks / 4) * 64 + 16 c + 4 (ks % 4) .. + 3.  qf: the factors that undo the
// powers of two of columns 2c and 2c + 1.
template <int D, bool WIDE, typename T>
__device__ __forceinline__ void f8_load_q(uint32_t (&qb)[D / 16][2], float (&qf)[2], const T *q, int rows, int lane) {
    const int head = WIDE ? lane >> 2 : (lane >> 2) & 3, c = lane & 3;
#pragma unroll
    for (int ks = 0; ks < D / 16; ks++) {
        uint2 v = make_uint2(0u, 0u);
        if (head < rows) v = *reinterpret_cast<const uint2 *>(q + head * D + (ks >> 2) * 64 + c * 16 + (ks & 3) * 4);
        qb[ks][0] = v.x;
        qb[ks][1] = v.y;
    }
    qf[0] = qf[1] = 1.f;
    if constexpr (!std::is_same<T, __half>::value) {
        float amax = 0.f;
#pragma unroll
        for (int ks = 0; ks < D / 16; ks++)
#pragma unroll
            for (int e = 0; e < 2; e++) {
                const float2 f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&qb[ks][e]));
                amax = fmaxf(amax, fmaxf(fabsf(f.x), fabsf(f.y)));
            }
        amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, 2));
        // the head's largest value goes to [2^14, 2^15): bf16's 8 bits then stay exact over 31 binades below it
        int sh = 14 - ((int)(__float_as_uint(amax) >> 23) - 127);
        sh = amax == 0.f || amax == INFINITY ? 0 : (sh > 100 ? 100 : sh);
        const float up = __uint_as_float((unsigned)(sh + 127) << 23);
#pragma unroll
        for (int ks = 0; ks < D / 16; ks++)
#pragma unroll
            for (int e = 0; e < 2; e++) {
                const float2 f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&qb[ks][e]));
                qb[ks][e] = Mma<__half>::pack(f.x * up, f.y * up);
            }
        const float down = __uint_as_float((unsigned)(127 - sh) << 23);
        qf[0] = __shfl_sync(kFull, down, (2 * c) * 4);
        qf[1] = __shfl_sync(kFull, down, (2 * c + 1) * 4);
    }
}

// TOK tokens (a multiple of 32) from row `base` of a stage.  sc: the stage's
// block scales (key scale * softmax scale * log2 e, value scale), a block per
// 2^log2_rows tokens.
template <int D, int TOK, bool WIDE, bool FULL>
__device__ __forceinline__ void f8_consume(const unsigned char *Ks, const unsigned char *Vs, const float2 *sc,
                                           int log2_rows, int base, int nvalid, int lane, int range,
                                           const uint32_t (&qb)[D / 16][2], const float (&qf)[2], F8State<D> &st) {
    constexpr int NG = TOK / 8;                  // groups of eight tokens
    const int n = lane >> 2, c = lane & 3;
    const int pn = perm_token<D>(n), pe = perm_token<D>(2 * c), po = perm_token<D>(2 * c + 1);
    // S^T = K Q^T: sixteen tokens (rows lane / 4 and + 8) at a time
    float x[NG][2], vs[NG];                      // this lane's tokens: row lane / 4 of the g-th group of eight
#pragma unroll
    for (int mt = 0; mt < NG / 2; mt++) {
        float s[4], s2[4];                       // two sums halve the chain of dependent products
#pragma unroll
        for (int e = 0; e < 4; e++) s[e] = s2[e] = 0.f;
        const int row = base + mt * 16 + pn;
#pragma unroll
        for (int k = 0; k < D / 64; k++) {
            const uint4 u = *reinterpret_cast<const uint4 *>(Ks + chunk_at<D>(row, c + 4 * k));
            const uint4 v = *reinterpret_cast<const uint4 *>(Ks + chunk_at<D>(row + 8, c + 4 * k));
            const uint32_t lo8[4] = {u.x, u.y, u.z, u.w}, hi8[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int ks = 0; ks < 4; ks++) {
                const uint32_t a[4] = {e4m3x2_lo(lo8[ks]), e4m3x2_lo(hi8[ks]), e4m3x2_hi(lo8[ks]),
                                       e4m3x2_hi(hi8[ks])};
                Mma<__half>::run((ks & 1) ? s2 : s, a, qb[4 * k + ks][0], qb[4 * k + ks][1]);
            }
        }
#pragma unroll
        for (int i = 0; i < 2; i++) {
            const int g = 2 * mt + i, tok = base + g * 8 + pn;
            const float2 f = sc[tok >> log2_rows];
            vs[g] = f.y;
#pragma unroll
            for (int e = 0; e < 2; e++) x[g][e] = (s[2 * i + e] + s2[2 * i + e]) * (qf[e] * f.x);
            if (!FULL && tok >= nvalid) {        // what stands past the context may be anything, its scales too
                x[g][0] = x[g][1] = -INFINITY;
                vs[g] = 0.f;
            }
        }
    }
    float mnew[2], alpha[2];
#pragma unroll
    for (int e = 0; e < 2; e++) {
        float mx = x[0][e];
#pragma unroll
        for (int g = 1; g < NG; g++) mx = fmaxf(mx, x[g][e]);
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, o));
        mnew[e] = fmaxf(st.m[e], mx);
        alpha[e] = ex2(st.m[e] - mnew[e]);
        st.m[e] = mnew[e];
    }
    float rnew[2], w[NG][2];
    if (!(range & 1)) {                                         // uniform over the warp
        const int top = range >> 1 > -100 ? range >> 1 : -100;
        const float wscale = __uint_as_float((unsigned)(kPExp - top + 127) << 23);
#pragma unroll
        for (int g = 0; g < NG; g++) w[g][0] = w[g][1] = vs[g] * wscale;
        rnew[0] = mnew[0] + (float)top;
        rnew[1] = mnew[1] + (float)top;
    } else {
#pragma unroll
        for (int e = 0; e < 2; e++) {
            float mx = -1e30f;                                  // finite: value scales of zero leave nothing
#pragma unroll
            for (int g = 0; g < NG; g++)
                if (vs[g] > 0.f && x[g][e] > -INFINITY) mx = fmaxf(mx, x[g][e] + log2f(vs[g]));
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, o));
            rnew[e] = fmaxf(st.r[e], mx);
#pragma unroll
            for (int g = 0; g < NG; g++)
                w[g][e] = vs[g] > 0.f ? fminf(exp2f(log2f(vs[g]) - (rnew[e] - mnew[e]) + (float)kPExp), 0x1p100f) : 0.f;
        }
    }
    // the probabilities, and P^T as B fragments
    uint32_t hi[NG], lo[NG];
#pragma unroll
    for (int g = 0; g < NG; g++) {
        const float p0 = ex2(x[g][0] - mnew[0]), p1 = ex2(x[g][1] - mnew[1]);
        st.l[0] = g == 0 ? fmaf(st.l[0], alpha[0], p0) : st.l[0] + p0;
        st.l[1] = g == 0 ? fmaf(st.l[1], alpha[1], p1) : st.l[1] + p1;
        const float w0 = p0 * w[g][0], w1 = p1 * w[g][1];
        uint32_t h = Mma<__half>::pack(w0, w1);
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h));
        const uint32_t rest = Mma<__half>::pack(w0 - f.x, w1 - f.y);
        if (WIDE) {
            hi[g] = transpose8x8(h);
            lo[g] = transpose8x8(rest);
        } else {
            hi[g] = transpose8x8(c < 2 ? h : rest);
        }
    }
    const float a0 = ex2(st.r[0] - rnew[0]), a1 = ex2(st.r[1] - rnew[1]);
    st.r[0] = rnew[0];
    st.r[1] = rnew[1];
    if (__any_sync(kFull, a0 != 1.f || a1 != 1.f)) {
#pragma unroll
        for (int i = 0; i < D / 16; i++) {
            st.o[i][0] *= a0;
            st.o[i][1] *= a1;
            st.o[i][2] *= a0;
            st.o[i][3] *= a1;
        }
    }
    // O^T += V^T P^T: sixteen tokens a step; rows lane / 4 and + 8 of tile i are d = (D / 8) (lane / 4) + 2 i and + 1
#pragma unroll
    for (int kt = 0; kt < NG / 2; kt++) {
        const int t = base + kt * 16;
        const int rows[4] = {t + pe, t + po, t + 8 + pe, t + 8 + po};
        uint32_t v[4][D / 32];
#pragma unroll
        for (int i = 0; i < 4; i++) {
            if constexpr (D >= 128) {
                const uint4 r = *reinterpret_cast<const uint4 *>(Vs + chunk_at<D>(rows[i], n));
                v[i][0] = r.x;
                v[i][1] = r.y;
                v[i][2] = r.z;
                v[i][3] = r.w;
            } else {
                const uint2 r = *reinterpret_cast<const uint2 *>(Vs + chunk_at<D>(rows[i], n >> 1) + (n & 1) * 8);
                v[i][0] = r.x;
                v[i][1] = r.y;
            }
        }
#pragma unroll
        for (int i = 0; i < D / 16; i++) {
            const uint32_t sel = (i & 1) ? 0x7362u : 0x5140u;   // bytes 2, 3 or 0, 1 of two tokens, interleaved
            const uint32_t x01 = __byte_perm(v[0][i >> 1], v[1][i >> 1], sel);
            const uint32_t x23 = __byte_perm(v[2][i >> 1], v[3][i >> 1], sel);
            const uint32_t a[4] = {e4m3x2_lo(x01), e4m3x2_hi(x01), e4m3x2_lo(x23), e4m3x2_hi(x23)};
            Mma<__half>::run(st.o[i], a, hi[2 * kt], hi[2 * kt + 1]);
            if (WIDE) Mma<__half>::run(st.o[i], a, lo[2 * kt], lo[2 * kt + 1]);
        }
    }
}

// A work item as the producer sees it.  ent holds, on lane j, block-table
// entry win + j of the sequence (-1 past its blocks), sc that block's scales.
struct F8Item {
    int s, part, nparts, g, h0, rows, tok0, ntok, nst, nblk, win, ent;
    float2 sc;
    int top, low;              // exponents of the value scales of the window's blocks, over the warp
};

// The scales of this lane's block, requested; f8_scale_range, when they are
// here, folds the softmax scale in and takes the window's exponents.
__device__ __forceinline__ float2 f8_load_scales(const F8Args &f, int g, int ent) {
    if (ent < 0 || ent >= f.a.num_blocks) return make_float2(0.f, -1.f);
    const float2 v = __ldg(f.scales + (size_t)ent * f.scale_heads + g);
    return make_float2(v.x * f.a.scale_log2, fmaxf(v.y, 0.f));
}

__device__ __forceinline__ void f8_scale_range(float2 sc, int &top, int &low) {
    const int e = exponent_above(sc.y);
    const int t = __reduce_max_sync(kFull, e);
    const int l = __reduce_min_sync(kFull, sc.y < 0.f ? 1000 : e);      // below zero: no block
    top = top > t ? top : t;
    low = low < l ? low : l;
}

template <int TOKENS>
__device__ __forceinline__ void f8_decode_item(const F8Args &f, const int *pref, const int *ctxs, int S, int tiles,
                                               unsigned int t, int lane, F8Item &it) {
    const AttnArgs &a = f.a;
    const int pidx = (int)(t / (unsigned int)tiles);
    const int tile = (int)(t % (unsigned int)tiles);
    int lo = 0, hi = S;                                            // pref[lo] <= pidx < pref[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (pref[mid] <= pidx) lo = mid; else hi = mid;
    }
    it.s = lo;
    it.part = pidx - pref[lo];
    it.nparts = pref[lo + 1] - pref[lo];
    it.g = tile / a.head_tiles;
    const int group = a.num_heads / a.num_kv_heads, first = (tile % a.head_tiles) * f.tile;
    it.h0 = it.g * group + first;
    it.rows = group - first < f.tile ? group - first : f.tile;
    const int ctx = ctxs[lo];
    it.tok0 = it.part * a.partition;
    const int ntok = ctx - it.tok0 < a.partition ? ctx - it.tok0 : a.partition;
    it.ntok = ntok < 0 ? 0 : ntok;
    it.nst = (it.ntok + TOKENS - 1) / TOKENS;
    it.nblk = (it.tok0 + it.ntok + (1 << a.log2_block) - 1) >> a.log2_block;      // blocks up to the item's end
    it.win = it.tok0 >> a.log2_block;
    const int j = it.win + lane;
    it.ent = j < it.nblk ? __ldg(a.tables + (size_t)lo * a.max_blocks + j) : -1;
}

// WIDE: items of five to eight query heads.
template <int D, bool WIDE, typename T>
__global__ void __launch_bounds__(kPipes * 64, kCtasPerSm)
    paged_attention_fp8_kernel(const F8Args f, const __grid_constant__ CUtensorMap tmk,
                               const __grid_constant__ CUtensorMap tmv) {
    using L = F8Layout;
    constexpr int R = L::R, TOKENS = kStageBytes / D;
    const AttnArgs &a = f.a;
    extern __shared__ __align__(1024) unsigned char smem8[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int pipe = warp & (kPipes - 1);
    unsigned char *ring = smem8 + L::rings + (uint32_t)pipe * L::q;                  // [R][2][TOKENS][D]
    unsigned char *rest = smem8 + L::rest + (uint32_t)pipe * L::rest_bytes - L::q;
    T *qs = reinterpret_cast<T *>(rest + L::q);                      // [8][D]
    float2 *scs = reinterpret_cast<float2 *>(rest + L::sc);          // [R][kStageBlocks]
    uint64_t *full = reinterpret_cast<uint64_t *>(rest + L::bars);
    uint64_t *empty = full + R;
    F8Meta *meta = reinterpret_cast<F8Meta *>(rest + L::meta);
    int &cta_flags = *reinterpret_cast<int *>(smem8 + L::misc);
    int *scan_tmp = reinterpret_cast<int *>(smem8 + L::misc) + 32;
    const int S = a.num_seqs;
    int *pref = reinterpret_cast<int *>(smem8 + L::seqs);            // [S + 1] partitions before s
    int *ctxs = pref + S + 1;                                        // [S]
    const int tiles = a.num_kv_heads * a.head_tiles;
    WsHeader *hdr = a.hdr;

    if (warp < kPipes && lane == 0) {
        for (int i = 0; i < R; i++) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        fence_mbar_init();
    }
    if (warp == kPipes && lane < 2) prefetch_tensor_map(lane ? &tmv : &tmk);
    pdl_trigger();
    pdl_wait();
    // every thread counts the partitions of its sequences, neighbouring ones, and what stands before them
    static_assert(kLaunchSeqs <= 2 * kPipes * 64, "two sequences to a thread");
    int ctx[2], parts[2];
#pragma unroll
    for (int i = 0; i < 2; i++) {
        const int q = 2 * (int)threadIdx.x + i;
        ctx[i] = q < S ? a.ctx_lens[q] : 0;
    }
    if (threadIdx.x == 0) {
        const unsigned magic = hdr->magic;
        cta_flags = (timed_out(a.st) ? 1 : 0) | (magic != kWsMagic8 ? 2 : 0) | ((smem_u32(smem8) & 1023u) ? 4 : 0);
    }
#pragma unroll
    for (int i = 0; i < 2; i++) {
        const int q = 2 * (int)threadIdx.x + i;
        if (ctx[i] < 0 || ctx[i] > a.max_ctx) {
            if (blockIdx.x == 0) latch(a.st, kFlagBadContext, ctx[i]);
            ctx[i] = ctx[i] < 0 ? 0 : a.max_ctx;
        }
        parts[i] = q >= S ? 0 : ctx[i] > 0 ? (ctx[i] + a.partition - 1) / a.partition : 1;
        if (q < S) ctxs[q] = ctx[i];
    }
    int upto = parts[0] + parts[1];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(kFull, upto, o);
        if (lane >= o) upto += y;
    }
    if (lane == 31) scan_tmp[warp] = upto;
    __syncthreads();
    if (cta_flags) {                                   // uniform over the CTA
        if ((cta_flags & 2) && blockIdx.x == 0 && threadIdx.x == 0) latch(a.st, kFlagBadWorkspace, hdr->magic);
        if ((cta_flags & 4) && blockIdx.x == 0 && threadIdx.x == 0) latch(a.st, kFlagTimeout, -2);
        return;
    }
#pragma unroll
    for (int w = 0; w < 2 * kPipes - 1; w++)
        if (w < warp) upto += scan_tmp[w];
    if (2 * (int)threadIdx.x < S) pref[2 * threadIdx.x + 1] = upto - parts[1];
    if (2 * (int)threadIdx.x + 1 < S) pref[2 * threadIdx.x + 2] = upto;
    if (threadIdx.x == 0) pref[0] = 0;
    __syncthreads();
    const unsigned int N = (unsigned int)pref[S] * (unsigned int)tiles;
    const int B = 1 << a.log2_block;
    constexpr int kLog2Tokens = TOKENS == 64 ? 6 : 5;
    const int log2_rows = a.log2_block < kLog2Tokens ? a.log2_block : kLog2Tokens;   // tokens per copy: a block, or a stage of it

    if (warp >= kPipes) {
        // ---------------- producer: tickets -> items -> tiled copies ----------------
        // At head_dim 128 the consumers' four warps take registers that these four give up: 72 + 184 =
        // 2 x 128, the launch's own (256 threads of 128, two CTAs to an SM).
        if constexpr (D >= 128) asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
        const T *qg = static_cast<const T *>(a.q);
        const int rows_per_copy = 1 << log2_rows;
        const int cps = TOKENS >> log2_rows;                         // blocks per stage
        const uint32_t copy_bytes = (uint32_t)rows_per_copy * D;
        // another head tile of the same kv head reads the same tiles next
        const uint64_t policy = a.head_tiles > 1 ? policy_evict_last() : policy_evict_first();
        // the first items go round the CTAs; later ones come from the counter
        const unsigned int pipes = gridDim.x * kPipes;
        unsigned int cur_t = (unsigned int)pipe * gridDim.x + blockIdx.x;
        F8Item cur, nx;
        if (cur_t < N) {
            f8_decode_item<TOKENS>(f, pref, ctxs, S, tiles, cur_t, lane, cur);
            cur.sc = f8_load_scales(f, cur.g, cur.ent);
        }
        int kk = 0, first = -R;                                      // stages so far, the last item's first one
        bool dead = false;
        while (cur_t < N && !dead) {
            // The next ticket is claimed three stages before the item's last, its table entries
            // are requested a stage later and their blocks' scales another stage later: each
            // has arrived when it is needed.
            unsigned int nxt_raw = 0, nxt_t = 0xffffffffu;
            int step = 0;                                            // claimed, decoded, scales requested
            auto next_item = [&]() {
                if (step == 0) {
                    if (lane == 0) nxt_raw = pipes + atomicAdd(&hdr->next, 1u);
                } else if (step == 1) {
                    nxt_t = __shfl_sync(kFull, nxt_raw, 0);
                    if (nxt_t < N) f8_decode_item<TOKENS>(f, pref, ctxs, S, tiles, nxt_t, lane, nx);
                } else {
                    if (nxt_t < N) nx.sc = f8_load_scales(f, nx.g, nx.ent);
                }
                step++;
            };
            const int npad = cur.nst > 0 ? cur.nst : 1;              // an empty context still has a stage
            const int32_t *trow = a.tables + (size_t)cur.s * a.max_blocks;
            const uint32_t q_bytes = (uint32_t)(cur.rows * D * 2);
            int win = cur.win, ent = cur.ent, top = -1000, low = 1000;
            float2 sc = cur.sc;
            f8_scale_range(sc, top, low);
            for (int i = 0; i < npad; i++, kk++) {
                if (i >= npad - 3) next_item();
                const int slot = kk % R;
                const bool withq = i == 0 && cur.nst > 0;
                int nv = 0, nb = 0, off0 = 0, pj = -1;
                float2 sj = make_float2(0.f, 0.f);
                if (i < cur.nst) {                                   // uniform over the warp
                    const int t_first = cur.tok0 + i * TOKENS;
                    const int lb0 = t_first >> a.log2_block;
                    off0 = t_first & (B - 1);
                    nv = cur.ntok - i * TOKENS < TOKENS ? cur.ntok - i * TOKENS : TOKENS;
                    nb = (nv + rows_per_copy - 1) >> log2_rows;
                    if (lb0 < win || lb0 + cps > win + 32) {
                        win = lb0;
                        const int j = win + lane;
                        ent = j < cur.nblk ? __ldg(trow + j) : -1;
                        sc = f8_load_scales(f, cur.g, ent);
                        f8_scale_range(sc, top, low);
                    }
                    const int jl = lane >> 1;                        // this lane's block of the stage
                    const int from = (lb0 + jl - win) & 31;
                    pj = __shfl_sync(kFull, ent, from);
                    sj.x = __shfl_sync(kFull, sc.x, from);
                    sj.y = __shfl_sync(kFull, sc.y, from);
                    const bool bad = jl < nb && (pj < 0 || pj >= a.num_blocks);
                    const unsigned badm = __ballot_sync(kFull, bad);
                    if (badm) {                                      // stop the stage at the first bad block
                        if (lane == __ffs(badm) - 1) latch(a.st, kFlagBadBlock, pj);
                        nb = (__ffs(badm) - 1) >> 1;
                        nv = nb << log2_rows;
                    }
                }
                bool ok = kk < R || mbar_wait(&empty[slot], ((kk / R) - 1) & 1, kWaitLimitCycles);
                // the one query buffer: the last item's first stage (which read it) must be consumed
                if (withq && first > kk - R) ok = ok && mbar_wait(&empty[first % R], (first / R) & 1, kWaitLimitCycles);
                if (!__all_sync(kFull, ok)) {
                    if (lane == 0) latch(a.st, kFlagTimeout, kk);
                    dead = true;
                    break;
                }
                if (i == 0) first = kk;
                if ((lane & 1) == 0 && (lane >> 1) < nb) scs[slot * kStageBlocks + (lane >> 1)] = sj;
                if (lane == 0) {
                    int4 *mv = reinterpret_cast<int4 *>(&meta[slot]);
                    mv[0] = make_int4(cur.s, cur.h0, cur.rows, cur.part);
                    mv[1] = make_int4(cur.nparts, nv, (i == 0 ? kFirst : 0) | (i == npad - 1 ? kLast : 0),
                                      scale_range(top, low));
                }
                __syncwarp();
                if (lane == 0)
                    mbar_arrive_expect_tx(&full[slot], 2u * copy_bytes * (uint32_t)nb + (withq ? q_bytes : 0u));
                __syncwarp();
                // lane 2j + t moves block j's K (t = 0) or V (t = 1) tile
                if (lane < 2 * nb) {
                    const int t = lane & 1;
                    unsigned char *dst = ring + (slot * 2 + t) * kStageBytes + (uint32_t)(lane >> 1) * copy_bytes;
                    tma_load_4d(dst, t ? (const void *)&tmv : (const void *)&tmk, 0, off0, cur.g, pj, &full[slot],
                                policy);
                }
                if (withq && lane == 0)
                    bulk_g2s(qs, qg + ((size_t)cur.s * a.num_heads + cur.h0) * D, q_bytes, &full[slot]);
            }
            if (dead) {                                              // copies may still be under way
                for (int k = kk < R ? 0 : kk - R; k < kk; k++) mbar_wait(&full[k % R], (k / R) & 1, kDrainLimitCycles);
                break;
            }
            while (step < 3) next_item();
            cur_t = nxt_t;
            cur = nx;
        }
        if (lane == 0) {
            if (!dead) {                                             // the stop mark
                const int slot = kk % R;
                if (kk >= R && !mbar_wait(&empty[slot], ((kk / R) - 1) & 1, kWaitLimitCycles)) {
                    latch(a.st, kFlagTimeout, kk);
                } else {
                    meta[slot].flags = kStop;
                    mbar_arrive_expect_tx(&full[slot], 0u);
                }
            }
            // the last pipeline to finish leaves the counters at zero for the next call
            __threadfence();
            if (atomicAdd(&hdr->done, 1u) == pipes - 1) {
                hdr->next = 0;
                hdr->done = 0;
                __threadfence();
            }
        }
        return;
    }

    // ---------------- consumer ----------------
    if constexpr (D >= 128) asm volatile("setmaxnreg.inc.sync.aligned.u32 184;");
    uint32_t qb[D / 16][2];
    float qf[2] = {1.f, 1.f};
    F8State<D> st;
    f8_reset(st);
    for (int k = 0;; k++) {
        const int slot = k % R;
        if (!__all_sync(kFull, mbar_wait(&full[slot], (k / R) & 1, kWaitLimitCycles))) {
            if (lane == 0) latch(a.st, kFlagTimeout, k);
            // what the producer has under way in the other slots
            for (int i = 1; i < R; i++) mbar_wait(&full[(k + i) % R], ((k + i) / R) & 1, kDrainLimitCycles);
            break;
        }
        const F8Meta md = meta[slot];
        if (md.flags & kStop) break;
        const unsigned char *Ks = ring + (slot * 2) * kStageBytes;
        unsigned char *Vs = ring + (slot * 2 + 1) * kStageBytes;
        const float2 *sc = scs + slot * kStageBlocks;
        if ((md.flags & kFirst) && md.nvalid > 0) f8_load_q<D, WIDE, T>(qb, qf, qs, md.rows, lane);
        if (md.nvalid == TOKENS) {
            f8_consume<D, TOKENS, WIDE, true>(Ks, Vs, sc, log2_rows, 0, TOKENS, lane, md.range, qb, qf, st);
        } else if (md.nvalid > 0) {
            // rows past the context may hold anything: zero them in V (0 * NaN would poison the sum)
            const int end = (md.nvalid + 31) & ~31;
            for (int v = md.nvalid * (D / 16) + lane; v < end * (D / 16); v += 32)
                reinterpret_cast<uint4 *>(Vs)[v] = make_uint4(0u, 0u, 0u, 0u);
            __syncwarp();
#pragma unroll 1
            for (int base = 0; base < md.nvalid; base += 32)
                f8_consume<D, 32, WIDE, false>(Ks, Vs, sc, log2_rows, base, md.nvalid, lane, md.range, qb, qf, st);
            fence_proxy_async_smem();            // the zeroed rows, before TMA refills the slot
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[slot]);
        if (!(md.flags & kLast)) continue;

        // ---- the item's end: this warp holds its whole state ----
        constexpr int W = D / 8;                 // this lane's d: W (lane / 4) .. + W - 1
        const int c = lane & 3;
#pragma unroll
        for (int e = 0; e < 2; e++) {
            float l = st.l[e];
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) l += __shfl_xor_sync(kFull, l, o);
            // o is relative to r - 15, the sum of exponentials to m
            const float rel = l > 0.f || l != l ? exp2f(st.r[e] - (float)kPExp - st.m[e]) : 0.f;
            float v[W];
#pragma unroll
            for (int i = 0; i < W / 2; i++) {
                v[2 * i] = st.o[i][e];
                v[2 * i + 1] = st.o[i][2 + e];
                if (!WIDE) {                     // the columns that carry the probabilities' rest
                    v[2 * i] += __shfl_xor_sync(kFull, v[2 * i], 2);
                    v[2 * i + 1] += __shfl_xor_sync(kFull, v[2 * i + 1], 2);
                }
                v[2 * i] *= rel;
                v[2 * i + 1] *= rel;
            }
            const int head = 2 * c + e;
            if (head >= md.rows || (!WIDE && c >= 2)) continue;
            const size_t sh = (size_t)md.s * a.num_heads + md.h0 + head;
            const int d0 = W * (lane >> 2);
            if (md.nparts <= 1) {
                const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
                uint4 *dst = reinterpret_cast<uint4 *>(static_cast<T *>(a.out) + sh * D + d0);
#pragma unroll
                for (int j = 0; j < W; j += 8)
                    dst[j / 8] = make_uint4(Mma<T>::pack(v[j] * inv, v[j + 1] * inv),
                                            Mma<T>::pack(v[j + 2] * inv, v[j + 3] * inv),
                                            Mma<T>::pack(v[j + 4] * inv, v[j + 5] * inv),
                                            Mma<T>::pack(v[j + 6] * inv, v[j + 7] * inv));
            } else {
                const size_t sp = sh * a.max_parts + md.part;
                float4 *dst = reinterpret_cast<float4 *>(a.ws_o + sp * D + d0);
#pragma unroll
                for (int j = 0; j < W; j += 4) dst[j / 4] = make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
                if (lane < 4) {                  // the merge takes a sum that is NaN for an empty one: v says it
                    a.ws_m[sp] = l != l ? 0.f : st.m[e];
                    a.ws_l[sp] = l != l ? 1.f : l;
                }
            }
        }
        f8_reset(st);
    }
}

// Merge the partitions of split contexts, a warp to a (sequence, head); for
// splits of up to 32 partitions (partition_reduce_kernel takes longer ones).
constexpr int kMergeThreads = 128;
constexpr int kMergeParts = 32;

template <int D, typename T> __global__ void __launch_bounds__(kMergeThreads) fp8_merge_kernel(const AttnArgs a) {
    pdl_trigger();
    pdl_wait();
    const int row = (int)((blockIdx.x * (unsigned)kMergeThreads + threadIdx.x) >> 5), lane = threadIdx.x & 31;
    if (row >= a.num_seqs * a.num_heads) return;
    const int s = row / a.num_heads;
    int ctx = a.ctx_lens[s];
    ctx = ctx < 0 ? 0 : ctx > a.max_ctx ? a.max_ctx : ctx;
    const int np = (ctx + a.partition - 1) / a.partition;
    if (np > 1) merge_partitions_warp<D, T>(a, s, row - s * a.num_heads, 1, np, lane);
}

__global__ void fp8_workspace_init_kernel(uint4 *ws, size_t n16) {
    pdl_trigger();
    pdl_wait();
    const size_t i = (size_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (i >= n16) return;
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    if (i == 0) v.z = kWsMagic8;                              // WsHeader: next, done, magic, pad
    if (i == kPrefillHeader / 16) v.z = kWsMagic;
    ws[i] = v;
}

// Tokens per partition.  A GPU of 152 SMs has 1216 pipelines (152 x kCtasPerSm x
// kPipes; the number is written down, since the workspace's size is asked for
// without a GPU and has to be the call's).  Where that many
// items hold everything, the shortest partitions that do so end first (1 x
// 8,000 tokens, 8 kv heads: 11.4 us at 64 tokens, 13.9 at 256); beyond, 256
// tokens (512 of head_dim 64) keep the items' beginnings and ends small beside
// them and their last round short (64 x up to 2,000 tokens, 8 kv heads: 30.0 us
// at 256, 32.5 at 128, 43.5 at 1024); and calls of so many items that rounds no
// longer matter take longer ones, which leave fewer partials (256 x up to 4,096
// tokens, 32 kv heads: 630 us at 1024, 659 at 256).
int choose_partition8(int partition_size, int num_seqs, int tiles, int head_dim, int max_ctx) {
    if (partition_size > 0) return partition_size;
    constexpr long long kPipelines = 152 * kCtasPerSm * kPipes;
    const long long n = (long long)num_seqs * tiles;
    for (int P = 64; P <= 256; P *= 2)
        if (n * parts_for(max_ctx, P) <= kPipelines) return P;
    int P = head_dim >= 128 ? 256 : 512;
    while (P < 1024 && n * parts_for(max_ctx, 2 * P) >= 24 * kPipelines) P *= 2;
    return P;
}

struct F8Sizes {
    int tile, head_tiles, P, MP;
    size_t m_off, l_off, o_off, bytes;
};

F8Sizes f8_sizes(int S, int H, int Hkv, int D, int max_ctx, int partition_size) {
    F8Sizes z;
    const int group = H / Hkv;
    z.head_tiles = (group + kTileHeads - 1) / kTileHeads;
    z.tile = (group + z.head_tiles - 1) / z.head_tiles;
    z.P = kernel_partition(choose_partition8(partition_size, S, Hkv * z.head_tiles, D, max_ctx), max_ctx, kMaxTokens);
    z.MP = parts_for(max_ctx, z.P);
    const size_t n = z.MP > 1 ? (size_t)S * H * z.MP : 0;
    z.m_off = kBodyOff;
    z.l_off = z.m_off + align256(n * sizeof(float));
    z.o_off = z.l_off + align256(n * sizeof(float));
    z.bytes = z.o_off + align256(n * D * sizeof(float));
    return z;
}

// The cache [NB][Hkv][B][D] of bytes as a 4-D tensor (innermost first); a box
// is whole rows of min(B, a stage's) tokens of one (block, kv head), swizzled.
bool encode_cache_map8(CUtensorMap *map, const void *base, int num_blocks, int Hkv, int B, int D) {
    PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
    if (!enc) return false;
    const cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)B, (cuuint64_t)Hkv, (cuuint64_t)(num_blocks > 0 ? num_blocks : 1)};
    const cuuint64_t strides[3] = {(cuuint64_t)D, (cuuint64_t)B * D, (cuuint64_t)Hkv * B * D};
    const cuuint32_t box[4] = {(cuuint32_t)D, (cuuint32_t)(B < kStageBytes / D ? B : kStageBytes / D), 1u, 1u};
    const cuuint32_t estr[4] = {1u, 1u, 1u, 1u};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<void *>(base), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, bool WIDE, typename T> cudaError_t launch_decode8w(const F8Args &f, cudaStream_t stream) {
    auto kern = paged_attention_fp8_kernel<D, WIDE, T>;
    const size_t smem = F8Layout::total(f.a.num_seqs);
    static std::atomic<unsigned long long> allowed{0};
    cudaError_t e = allow_smem(kern, F8Layout::total(kLaunchSeqs), allowed);
    if (e != cudaSuccess) return e;
    CUtensorMap tmk, tmv;
    const AttnArgs &a = f.a;
    if (!encode_cache_map8(&tmk, a.k_cache, a.num_blocks, a.num_kv_heads, 1 << a.log2_block, D) ||
        !encode_cache_map8(&tmv, a.v_cache, a.num_blocks, a.num_kv_heads, 1 << a.log2_block, D))
        return cudaErrorInvalidValue;
    const long long items = (long long)a.num_seqs * a.max_parts * a.num_kv_heads * a.head_tiles;
    long long ctas = (long long)sm_count() * kCtasPerSm;
    if (ctas > items) ctas = items;                  // few items: one to a CTA
    return launch(kern, dim3((unsigned)ctas), dim3(kPipes * 64), smem, stream, f, tmk, tmv);
}

template <int D, typename T> cudaError_t launch_decode8(const F8Args &f, cudaStream_t stream) {
    cudaError_t e = f.tile > 4 ? launch_decode8w<D, true, T>(f, stream) : launch_decode8w<D, false, T>(f, stream);
    if (e != cudaSuccess || f.a.max_parts <= 1) return e;
    const unsigned rows = (unsigned)f.a.num_seqs * (unsigned)f.a.num_heads;      // <= kLaunchSeqs heads
    if (f.a.max_parts <= kMergeParts)
        return launch(fp8_merge_kernel<D, T>, dim3((rows + kMergeThreads / 32 - 1) / (kMergeThreads / 32)),
                      dim3(kMergeThreads), 0, stream, f.a);
    return launch_reduce<T>(D, f.a, dim3((unsigned)f.a.num_heads, (unsigned)f.a.num_seqs), stream);
}

// ---- the prompt phase ------------------------------------------------------------

// Logical block j of sequence s, as 16-bit values, to block s * width + j of a
// scratch pool of the same layout; new_tables names those blocks.  A code
// times a power of two is exact in bf16, and in fp16 within its range (times
// another scale it is rounded).  Rows past the context become zeros.  A full block that an earlier sequence holds
// in the same place (a shared prefix) is widened there once and named by both
// (32 requests after a shared 1000-token prefix: 358 us the whole call without
// that).  One CTA per block, eight codes of K and of V to a load: bound by
// the bytes read and twice as many written.
constexpr int kWidenThreads = 256;
constexpr int kWidenUnroll = 4;

// Keys enter fp16 at half their size (the softmax scale makes up for it), so that
// rotated keys of fp16 inputs, up to 65504 sqrt(2), stay in its range.
template <typename T> constexpr float kKeyFactor = std::is_same<T, __half>::value ? 0.5f : 1.f;

// Two fp32 to one register of two 16-bit numbers (x in the low half), to nearest
// even, clamped at the largest number, NaN to NaN: what is finite in the cache
// stays finite (an fp16 value of 65504 is 65536 in 8 bits).  An infinite value would
// give NaN in earlier rows of its key tile, where its probability is 0.
template <typename T> __device__ __forceinline__ uint32_t pack_finite(float x, float y) {
    uint32_t d;
    if constexpr (std::is_same<T, __half>::value)
        asm("cvt.rn.satfinite.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(y), "f"(x));
    else
        asm("cvt.rn.satfinite.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(y), "f"(x));
    return d;
}

template <typename T> __device__ __forceinline__ uint4 widen8(const uint2 &w, float s) {
    const uint32_t in[2] = {w.x, w.y};
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 2; i++) {
        const uint32_t lo = e4m3x2_lo(in[i]), hi = e4m3x2_hi(in[i]);
        const float2 x = __half22float2(*reinterpret_cast<const __half2 *>(&lo));
        const float2 y = __half22float2(*reinterpret_cast<const __half2 *>(&hi));
        o[2 * i] = pack_finite<T>(x.x * s, x.y * s);
        o[2 * i + 1] = pack_finite<T>(y.x * s, y.y * s);
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}

template <typename T>
__global__ void __launch_bounds__(kWidenThreads) widen_blocks_kernel(
    uint4 *__restrict__ k_out, uint4 *__restrict__ v_out, int32_t *__restrict__ new_tables, const WsHeader *hdr,
    const uint2 *__restrict__ k_cache, const uint2 *__restrict__ v_cache, const float2 *__restrict__ scales,
    const int32_t *__restrict__ tables, const int32_t *__restrict__ ctx_lens, int width, int max_blocks, int log2_block,
    int num_blocks, int num_kv_heads, int row_chunks, DeviceStatus *st) {
    pdl_trigger();
    pdl_wait();
    if (hdr->magic != kWsMagic8) {
        if (blockIdx.x == 0 && threadIdx.x == 0) latch(st, kFlagBadWorkspace, hdr->magic);
        return;
    }
    const int s = (int)(blockIdx.x / (unsigned)width), j = (int)(blockIdx.x % (unsigned)width);
    const int B = 1 << log2_block;
    const int rows = ctx_lens[s] - (j << log2_block);                // tokens of the context in this block and after
    const bool inside = rows > 0 && j < max_blocks;
    const int32_t b = inside ? tables[(size_t)s * max_blocks + j] : -1;
    const bool good = b >= 0 && b < num_blocks;
    // the first sequence that holds this block, full, in this place; every warp finds the same one
    int owner = s;
    if (good && rows >= B) {
        for (int base = 0; base < s; base += 32) {
            const int q = base + (threadIdx.x & 31);
            const bool same = q < s && tables[(size_t)q * max_blocks + j] == b && ctx_lens[q] >= ((j + 1) << log2_block);
            const unsigned m = __ballot_sync(kFull, same);
            if (m) {
                owner = base + __ffs(m) - 1;
                break;
            }
        }
    }
    if (threadIdx.x == 0) new_tables[blockIdx.x] = owner * width + j;
    if (inside && !good && threadIdx.x == 0) latch(st, kFlagBadBlock, b);
    if (!good || owner != s) return;
    // eight-code chunks of a (block, head); a row's are 8 or 16
    const int log2_row = row_chunks == 16 ? 4 : 3, log2_head = log2_row + log2_block;
    const int chunks = num_kv_heads << log2_head;
    const float2 *sc = scales + (size_t)b * scale_heads(num_kv_heads);
    const uint2 *kin = k_cache + (size_t)b * chunks, *vin = v_cache + (size_t)b * chunks;
    uint4 *ko = k_out + (size_t)blockIdx.x * chunks, *vo = v_out + (size_t)blockIdx.x * chunks;
    // four chunks of each at a time under way
    for (int i0 = threadIdx.x; i0 < chunks; i0 += kWidenThreads * kWidenUnroll) {
        uint2 kw[kWidenUnroll], vw[kWidenUnroll];
        float2 f[kWidenUnroll];
#pragma unroll
        for (int k = 0; k < kWidenUnroll; k++) {
            const int i = i0 + k * kWidenThreads;
            if (i < chunks) {
                kw[k] = kin[i];
                vw[k] = vin[i];
                f[k] = sc[i >> log2_head];
            }
        }
#pragma unroll
        for (int k = 0; k < kWidenUnroll; k++) {
            const int i = i0 + k * kWidenThreads;
            if (i >= chunks) break;
            const bool past = rows < B && ((i & ((1 << log2_head) - 1)) >> log2_row) >= rows;
            ko[i] = past ? make_uint4(0u, 0u, 0u, 0u) : widen8<T>(kw[k], f[k].x * kKeyFactor<T>);
            vo[i] = past ? make_uint4(0u, 0u, 0u, 0u) : widen8<T>(vw[k], f[k].y);
        }
    }
}

struct WidenSizes {
    int width;                   // blocks per sequence
    size_t k_off, v_off, bytes;
};

WidenSizes widen_sizes(int S, int Hkv, int D, int B, int max_ctx) {
    WidenSizes z;
    z.width = (int)(((long long)max_ctx + B - 1) / B);
    const size_t blocks = (size_t)S * z.width;
    z.k_off = kBodyOff + align256(blocks * sizeof(int32_t));
    z.v_off = z.k_off + align256(blocks * Hkv * B * D * 2);
    z.bytes = z.v_off + align256(blocks * Hkv * B * D * 2);
    return z;
}

// What both calls ask of the cache.
pkv_status check_cache8(const char *what, int num_heads, int num_kv_heads, int head_dim, int block_size,
                        pkv_dtype dtype) {
    if (dtype != PKV_F16 && dtype != PKV_BF16) return fail(PKV_EINVAL, "%s: bad dtype %d", what, (int)dtype);
    if (head_dim != 64 && head_dim != 128)
        return fail(PKV_EINVAL, "%s: head_dim %d not supported (64 or 128)", what, head_dim);
    if (!is_pow2(block_size) || block_size < kMinBlock || block_size > 128)
        return fail(PKV_EINVAL, "%s: block_size %d not a power of two in [4, 128]", what, block_size);
    if (num_heads <= 0 || num_kv_heads <= 0 || num_heads % num_kv_heads || num_heads > 65535)
        return fail(PKV_EINVAL, "%s: %d query heads do not group over %d kv heads", what, num_heads, num_kv_heads);
    return PKV_OK;
}

}  // namespace
}  // namespace pkv

extern "C" {

pkv_status paged_attention_fp8_workspace_init(void *workspace, size_t workspace_bytes, struct CUstream_st *stream) {
    using namespace pkv;
    if (!workspace || workspace_bytes < kBodyOff || !aligned16(workspace))
        return fail(PKV_EINVAL, "paged_attention_fp8_workspace_init: need a 16-byte aligned workspace of at least %zu bytes",
                    kBodyOff);
    const size_t n16 = kBodyOff / 16;
    cudaError_t e = launch(fp8_workspace_init_kernel, dim3((unsigned)((n16 + 255) / 256)), dim3(256), 0, stream,
                           static_cast<uint4 *>(workspace), n16);
    if (e != cudaSuccess) return fail(PKV_ECUDA, "paged_attention_fp8_workspace_init: launch: %s", cudaGetErrorString(e));
    return PKV_OK;
}

size_t paged_attention_decode_fp8_workspace_size(int num_seqs, int num_heads, int num_kv_heads, int head_dim,
                                                 int max_context_len, int partition_size) {
    if (num_seqs <= 0 || num_heads <= 0 || num_kv_heads <= 0 || num_heads % num_kv_heads || head_dim <= 0 ||
        max_context_len < 0 || partition_size < 0)
        return 0;
    return pkv::f8_sizes(num_seqs, num_heads, num_kv_heads, head_dim, max_context_len, partition_size).bytes;
}

pkv_status paged_attention_decode_fp8(void *out, const void *query, const void *key_cache, const void *value_cache,
                                      const float *scales, const int32_t *block_tables, const int32_t *context_lens,
                                      int num_seqs, int max_blocks_per_seq, int max_context_len, int block_size,
                                      int num_blocks, int num_heads, int num_kv_heads, int head_dim, float scale,
                                      int partition_size, void *workspace, size_t workspace_bytes, pkv_dtype dtype,
                                      struct CUstream_st *stream) {
    using namespace pkv;
    const char *what = "paged_attention_decode_fp8";
    const pkv_status ok = check_cache8(what, num_heads, num_kv_heads, head_dim, block_size, dtype);
    if (ok != PKV_OK) return ok;
    if (num_seqs < 0 || num_seqs > 65535 || max_blocks_per_seq < 0 || num_blocks < 0)
        return fail(PKV_EINVAL, "%s: bad sizes (seqs %d, table width %d, blocks %d)", what, num_seqs, max_blocks_per_seq,
                    num_blocks);
    if (partition_size < 0 || partition_size % kMaxTokens)
        return fail(PKV_EINVAL, "%s: partition_size %d not a multiple of %d", what, partition_size, kMaxTokens);
    if (!std::isfinite(scale)) return fail(PKV_EINVAL, "%s: scale must be finite", what);
    const int64_t table_cap = (int64_t)max_blocks_per_seq * block_size;
    if (max_context_len < 0 || max_context_len > table_cap)
        return fail(PKV_EINVAL, "%s: max_context_len %d beyond the table (%lld tokens)", what, max_context_len,
                    (long long)table_cap);
    if (num_seqs == 0) return PKV_OK;
    // contexts of 2^30 tokens and more are latched as beyond their bound: the kernel rounds lengths up in 31 bits
    const int64_t bound = max_context_len > 0 ? max_context_len : table_cap;
    const int max_ctx = (int)(bound > INT32_MAX / 2 ? INT32_MAX / 2 : bound);
    if (!out || !query || !key_cache || !value_cache || !scales || !block_tables || !context_lens)
        return fail(PKV_EINVAL, "%s: NULL pointer", what);
    if (!aligned16(out) || !aligned16(query) || !aligned16(key_cache) || !aligned16(value_cache) || !aligned16(scales))
        return fail(PKV_EINVAL, "%s: pointers must be 16-byte aligned", what);
    const F8Sizes z = f8_sizes(num_seqs, num_heads, num_kv_heads, head_dim, max_ctx, partition_size);
    if (z.MP > 65535 || (long long)num_seqs * z.MP * num_kv_heads * z.head_tiles > INT_MAX / 2)
        return fail(PKV_EINVAL, "%s: %d partitions per sequence", what, z.MP);
    if (!workspace || workspace_bytes < z.bytes || !aligned16(workspace))
        return fail(PKV_EINVAL, "%s: workspace of %zu bytes needed, %zu given", what, z.bytes,
                    workspace ? workspace_bytes : (size_t)0);
    DeviceStatus *st = status_ptr();
    if (!st) return fail(PKV_ECUDA, "%s: no device status word", what);
    unsigned char *ws = static_cast<unsigned char *>(workspace);
    F8Args f;
    std::memset(&f, 0, sizeof f);
    AttnArgs &a = f.a;
    a.hdr = reinterpret_cast<WsHeader *>(ws);
    a.k_cache = key_cache;
    a.v_cache = value_cache;
    a.st = st;
    a.max_blocks = max_blocks_per_seq;
    a.max_ctx = max_ctx;
    a.log2_block = ilog2(block_size);
    a.num_blocks = num_blocks;
    a.num_heads = num_heads;
    a.num_kv_heads = num_kv_heads;
    a.head_tiles = z.head_tiles;
    a.partition = z.P;
    a.max_parts = z.MP;
    a.scale_log2 = scale * kLog2e;
    f.scales = reinterpret_cast<const float2 *>(scales);
    f.scale_heads = scale_heads(num_kv_heads);
    f.tile = z.tile;
    const size_t row = (size_t)num_heads * head_dim;
    for (int s0 = 0; s0 < num_seqs; s0 += kLaunchSeqs) {
        const int S = num_seqs - s0 < kLaunchSeqs ? num_seqs - s0 : kLaunchSeqs;
        a.num_seqs = S;
        a.out = static_cast<unsigned char *>(out) + s0 * row * 2;
        a.q = static_cast<const unsigned char *>(query) + s0 * row * 2;
        a.tables = block_tables + (size_t)s0 * max_blocks_per_seq;
        a.ctx_lens = context_lens + s0;
        const size_t part = (size_t)s0 * num_heads * z.MP;
        a.ws_m = reinterpret_cast<float *>(ws + z.m_off) + part;
        a.ws_l = reinterpret_cast<float *>(ws + z.l_off) + part;
        a.ws_o = reinterpret_cast<float *>(ws + z.o_off) + part * head_dim;
        cudaError_t e;
        if (head_dim == 128)
            e = dtype == PKV_F16 ? launch_decode8<128, __half>(f, stream) : launch_decode8<128, __nv_bfloat16>(f, stream);
        else
            e = dtype == PKV_F16 ? launch_decode8<64, __half>(f, stream) : launch_decode8<64, __nv_bfloat16>(f, stream);
        if (e != cudaSuccess) return fail(PKV_ECUDA, "%s: launch: %s", what, cudaGetErrorString(e));
    }
    return PKV_OK;
}

size_t paged_attention_prefill_fp8_workspace_size(int num_seqs, int num_kv_heads, int head_dim, int block_size,
                                                  int max_context_len) {
    if (num_seqs <= 0 || num_kv_heads <= 0 || head_dim <= 0 || block_size <= 0 || max_context_len < 0) return 0;
    return pkv::widen_sizes(num_seqs, num_kv_heads, head_dim, block_size, max_context_len).bytes;
}

pkv_status paged_attention_prefill_fp8(void *out, const void *query, const void *key_cache, const void *value_cache,
                                       const float *scales, const int32_t *block_tables, const int32_t *context_lens,
                                       const int32_t *query_start, int num_seqs, int num_tokens, int max_query_len,
                                       int max_context_len, int max_blocks_per_seq, int block_size, int num_blocks,
                                       int num_heads, int num_kv_heads, int head_dim, float scale, void *workspace,
                                       size_t workspace_bytes, pkv_dtype dtype, struct CUstream_st *stream) {
    using namespace pkv;
    const char *what = "paged_attention_prefill_fp8";
    const pkv_status ok = check_cache8(what, num_heads, num_kv_heads, head_dim, block_size, dtype);
    if (ok != PKV_OK) return ok;
    if (num_seqs < 0 || num_seqs > 65535 || num_tokens < 0 || max_query_len < 0 || num_blocks < 0)
        return fail(PKV_EINVAL, "%s: bad sizes (seqs %d, tokens %d, max query length %d, blocks %d)", what, num_seqs,
                    num_tokens, max_query_len, num_blocks);
    const float wide_scale = scale / (dtype == PKV_F16 ? kKeyFactor<__half> : kKeyFactor<__nv_bfloat16>);
    if (!(scale > 0.f) || wide_scale == INFINITY)
        return fail(PKV_EINVAL, "%s: scale must be positive and finite (for fp16 twice as well)", what);
    const int64_t table_cap = (int64_t)max_blocks_per_seq * block_size;
    if (max_blocks_per_seq < 0 || table_cap > INT_MAX || max_context_len < 0 || max_context_len > table_cap)
        return fail(PKV_EINVAL, "%s: max_context_len %d beyond the table (%lld tokens)", what, max_context_len,
                    (long long)table_cap);
    if (num_seqs == 0 || num_tokens == 0) return PKV_OK;
    const int max_ctx = max_context_len > 0 ? max_context_len : (int)table_cap;
    if (max_ctx <= 0 || num_blocks <= 0)
        return fail(PKV_EINVAL, "%s: num_blocks %d / table width %d not positive", what, num_blocks, max_blocks_per_seq);
    if (!out || !query || !key_cache || !value_cache || !scales || !block_tables || !context_lens || !query_start)
        return fail(PKV_EINVAL, "%s: NULL pointer", what);
    if (!aligned16(out) || !aligned16(query) || !aligned16(key_cache) || !aligned16(value_cache) || !aligned16(scales))
        return fail(PKV_EINVAL, "%s: pointers must be 16-byte aligned", what);
    const WidenSizes z = widen_sizes(num_seqs, num_kv_heads, head_dim, block_size, max_ctx);
    if ((long long)num_seqs * z.width > INT_MAX)
        return fail(PKV_EINVAL, "%s: %lld blocks of context", what, (long long)num_seqs * z.width);
    // all that the second call would refuse is refused here, before the first one launches
    const long long items = prefill_items(num_seqs, num_tokens, max_query_len, num_heads, num_kv_heads);
    if (items > kMaxPrefillItems)
        return fail(PKV_EINVAL, "%s: %lld work items (query tile pairs x heads x sequences) above 2^30", what, items);
    if (!workspace || workspace_bytes < z.bytes || !aligned16(workspace))
        return fail(PKV_EINVAL, "%s: workspace of %zu bytes needed, %zu given", what, z.bytes,
                    workspace ? workspace_bytes : (size_t)0);
    DeviceStatus *st = status_ptr();
    if (!st) return fail(PKV_ECUDA, "%s: no device status word", what);
    unsigned char *ws = static_cast<unsigned char *>(workspace);
    int32_t *new_tables = reinterpret_cast<int32_t *>(ws + kBodyOff);
    const int blocks = num_seqs * z.width;
    auto widen = dtype == PKV_F16 ? widen_blocks_kernel<__half> : widen_blocks_kernel<__nv_bfloat16>;
    cudaError_t e = launch(widen, dim3((unsigned)blocks), dim3(kWidenThreads), 0, stream,
                           reinterpret_cast<uint4 *>(ws + z.k_off), reinterpret_cast<uint4 *>(ws + z.v_off), new_tables,
                           reinterpret_cast<const WsHeader *>(ws), static_cast<const uint2 *>(key_cache),
                           static_cast<const uint2 *>(value_cache), reinterpret_cast<const float2 *>(scales), block_tables,
                           context_lens, z.width, max_blocks_per_seq, ilog2(block_size), num_blocks, num_kv_heads,
                           head_dim / 8, st);
    if (e != cudaSuccess) return fail(PKV_ECUDA, "%s: launch: %s", what, cudaGetErrorString(e));
    return paged_attention_prefill(out, query, ws + z.k_off, ws + z.v_off, new_tables, context_lens, query_start, num_seqs,
                                   num_tokens, max_query_len, z.width, block_size, blocks, num_heads, num_kv_heads,
                                   head_dim, wide_scale, ws + kPrefillHeader, kWsHeaderBytes, dtype, stream);
}

}  // extern "C"
