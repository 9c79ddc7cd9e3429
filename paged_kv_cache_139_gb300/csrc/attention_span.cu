// Decode attention over spans of a paged context: a sliding window with first
// tokens that stay visible (sinks), and sequences that share a prefix.
//
// What it computes.  A query row sees a set of its context's tokens; with
// x_t = scale * q . K_t over them,  out = sum_t softmax(x)_t V_t.
//   window  a sequence of n tokens sees [0, min(sinks, n)) and [n - window, n)
//   shared  it sees all n, in two halves: its own tokens [prefix, n), and the
//           prefix, computed once for all sequences of its group.  Each half is
//           (m, l, o) = (max x, sum 2^(x - m), sum 2^(x - m) V) in the log2
//           domain, and halves join as M = max m, sum l 2^(m - M), sum o 2^(m - M).
//
// What bounds it: HBM, at 2 d operations per key and query row against 2 d
// bytes.  So the work goes by (sequence or group, kv head): every key and value
// is read once for all query rows that see it.
//
// How (sm_103a):
//   * One CTA of two or four warps per (sequence, kv head), with 8 or 16 query heads as
//     the columns of S^T = K Q^T and O^T = V^T P^T (mma.sync m16n8k16): the
//     tokens are the 16-row operand, so one head or eight cost the same.  The
//     fifth-generation tensor cores would want 64 rows of queries; four heads
//     do not fill them, and at 48 products per 16 KB they are not what bounds.
//   * Each warp streams stages of 16 tokens through a ring of its own (16 KB): it
//     issues its tiled TMA copies itself and refills a slot as soon as it has
//     read it, so no warp waits for another before the end.
//   * Probabilities enter the second product as a rounded part and its
//     remainder (22 bits in fp16, 16 in bf16): rounded once they would add an
//     error as large as the output's own rounding.
//   * Invisible tokens of a stage (past the context, before the window, between
//     sinks and window) get -inf scores and zeroed value fragments; blocks that
//     hold none but those are not read, nor are their table entries.
//   * Few sequences are spread over the GPU by clusters of 2 to 16 CTAs per
//     (sequence, kv head), which join through distributed shared memory: no
//     workspace, no second launch, no counters.
//   * The shared form: groups of few query rows per kv head (up to 16, or more
//     over short prefixes) take their prefix through this kernel too, and the
//     launch for own tokens overlaps that one's end, joining the two halves
//     itself.  Larger groups go to the tcgen05 kernel, which takes some of the SMs while own tokens, bound by
//     memory, take the others; a third launch joins.
//
// Measured on one GB300: 256 sequences of up to 4,096 tokens, window 1,024, 32 heads:
// 7.42 TB/s (483 us; the copy rate is 6.79); 48 of up to 32,768, window 4,096, 32/8
// heads: 6.8 TB/s; 64 of the OPT-13B layer, window 255: 6.2 TB/s (43 us, of which
// start and tail some 5); one sequence, window 4,096, 32/8 heads: 8.8 us; four small
// ones 3.4 us.  Shared: 64 x 4 samples 161 us (6.8 TB/s over what is read once).
// Under ncu the tensor pipe is 13 % and issue slots 23 % busy on the OPT-13B batch.
// Tried and not kept: CTAs of one warp (8,192 items of 64 tokens 56 against 59 us, but
// 64 x 2,048 96 against 83); rings twice as deep where each CTA has an SM to itself
// (one sequence 14.9 against 8.6 us: clusters of 16 no longer fit beside one another);
// a cluster's CTAs reading one another's parts instead of writing them (9.7 us).
#include <cuda.h>

#include <algorithm>
#include <cmath>
#include <cstring>

#include "pkv_attention.cuh"
#include "pkv_host.cuh"
#include "pkv_span.cuh"
#include "pkv_tmap.h"

namespace pkv {
namespace {

constexpr int kTok = 16;                       // tokens of a stage: the rows of one product
constexpr int kFine = 4;                       // tokens of the small boxes
constexpr int kMaxCluster = 16;

// What a launch computes: a window; a prefix (to memory); own tokens, joined with the prefix's parts at
// the end; or own tokens as one part more, which a third launch joins with the others.
enum SpanMode { kSpanWindow, kSpanPrefix, kSpanSuffix, kSpanOwn };

struct SpanArgs {
    void *out;                   // [S][H][D]
    const void *q;               // [S][H][D]
    const int32_t *tables;       // [S][max_blocks]
    const int32_t *ctx_lens;     // [S]
    const int32_t *prefix_lens;  // [S]     shared
    const int32_t *group_start;  // [groups + 1]
    DeviceStatus *st;
    int num_seqs, num_groups, max_blocks, max_ctx, max_prefix, max_group;
    int log2_block, num_blocks, num_heads, num_kv_heads;
    int group;                   // query heads per kv head
    int head_tiles, tile_heads;  // a kv head's query heads in tiles of at most 8 NT
    int window, sinks;
    int fine;                    // stages with invisible tokens come in boxes of four tokens, as far as they are seen
    float scale_log2;
    PrefixParts parts;
};

// W warps per CTA (2 or 4), R ring slots per warp, CTAS resident CTAs per SM.
template <int D, int NT, int W> struct SpanConf {
    static constexpr int THREADS = W * 32;
    static constexpr int HALVES = D / 64;
    static constexpr uint32_t HALF_BYTES = kTok * 128;                 // 16 tokens x 64 elements
    static constexpr uint32_t TENSOR_BYTES = HALVES * HALF_BYTES;
    static constexpr uint32_t STAGE_BYTES = 2 * TENSOR_BYTES;
    static constexpr int R = D == 128 ? 2 : 4;
    static constexpr int CTAS = (NT == 1 ? 12 : 8) / W;
    static constexpr int COLS = 8 * NT;
    static constexpr int LD = D + 4;                                   // fp32 row of an output: 8 columns apart on 8 banks
    static constexpr uint32_t ring_bytes = R * STAGE_BYTES;            // a warp's, from offset 0 on
    static constexpr uint32_t wml = W * ring_bytes;                    // the warps' m, l [W][2][COLS]
    static constexpr uint32_t bars = wml + W * 2 * COLS * 4;
    static constexpr uint32_t got = bars + W * R * 8;                  // parts from the cluster's CTAs (CTAs of four warps):
    static constexpr int GOT = COLS * D / 4 + kMaxCluster;             // units of four elements, o [GOT][4] and m, l [GOT][2]
    static constexpr uint32_t got_ml = got + GOT * 16;
    static constexpr uint32_t bytes = W == 4 ? got_ml + GOT * 8 : got;
    static_assert(COLS * LD * 4 <= ring_bytes, "a warp's outputs fit its ring");
    static_assert(bars % 8 == 0 && got % 16 == 0 && got_ml % 8 == 0, "alignment");
};

__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// 2^x by the hardware approximation; 2^-inf = 0.
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Two fp32 as a rounded 16-bit pair and the pair of what the rounding left.
template <typename T> __device__ __forceinline__ void split_pair(float x, float y, uint32_t &hi, uint32_t &lo);
template <> __device__ __forceinline__ void split_pair<__half>(float x, float y, uint32_t &hi, uint32_t &lo) {
    const __half2 h = __floats2half2_rn(x, y);
    const float2 f = __half22float2(h);
    hi = *reinterpret_cast<const uint32_t *>(&h);
    lo = Mma<__half>::pack(x - f.x, y - f.y);
}
template <> __device__ __forceinline__ void split_pair<__nv_bfloat16>(float x, float y, uint32_t &hi, uint32_t &lo) {
    hi = Mma<__nv_bfloat16>::pack(x, y);
    lo = Mma<__nv_bfloat16>::pack(x - __uint_as_float(hi << 16), y - __uint_as_float(hi & 0xffff0000u));
}

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
// The shared address of CTA `rank` of the cluster that corresponds to this CTA's `addr`.
__device__ __forceinline__ uint32_t map_rank(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
__device__ __forceinline__ void st_cluster4(uint32_t addr, const float4 &v) {
    asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w)
                 : "memory");
}
__device__ __forceinline__ void st_cluster2(uint32_t addr, float x, float y) {
    asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(addr), "f"(x), "f"(y) : "memory");
}

// A running (m, l, o) of four output elements, and another part joined to it.
struct Joined {
    float m, l;
    float4 o;
    __device__ __forceinline__ void add(float m2, float l2, const float4 &o2) {
        // (parts that saw no token have weight 0 and values 0; a NaN score leaves m alone and shows in l and o)
        const float M = fmaxf(m, m2), z = M == -INFINITY ? 0.f : M;
        const float a = ex2(m - z), b = ex2(m2 - z);
        m = M;
        l = l * a + l2 * b;
        o.x = o.x * a + o2.x * b;
        o.y = o.y * a + o2.y * b;
        o.z = o.z * a + o2.z * b;
        o.w = o.w * a + o2.w * b;
    }
};

template <int D, int NT, int W, typename T, int MODE>
__global__ void __launch_bounds__(SpanConf<D, NT, W>::THREADS, SpanConf<D, NT, W>::CTAS)
    span_attention_kernel(const SpanArgs a, const __grid_constant__ CUtensorMap tmk,
                          const __grid_constant__ CUtensorMap tmv, const __grid_constant__ CUtensorMap tmk4,
                          const __grid_constant__ CUtensorMap tmv4) {
    using C = SpanConf<D, NT, W>;
    constexpr bool kClusters = W == 4 && (MODE == kSpanWindow || MODE == kSpanSuffix);
    constexpr bool kFineBoxes = D == 128 && MODE != kSpanPrefix;
    constexpr int R = C::R, HALVES = C::HALVES, COLS = C::COLS, LD = C::LD;
    // the 128-byte swizzle repeats every 1024 bytes: the ring starts on such a boundary
    extern __shared__ __align__(1024) unsigned char smem_span[];
    unsigned char *sm = smem_span;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t nrank = kClusters ? cluster_size() : 1u, rank = kClusters ? cluster_rank() : 0u;
    uint64_t *full = reinterpret_cast<uint64_t *>(sm + C::bars) + warp * R;      // this warp's own
    unsigned char *ring = sm + warp * C::ring_bytes;
    if (lane == 0) {
        for (int i = 0; i < R; i++) mbar_init(&full[i], 1);
        fence_mbar_init();
        if (warp == 0) {
            prefetch_tensor_map(&tmk);
            prefetch_tensor_map(&tmv);
            if (kFineBoxes && a.fine) {
                prefetch_tensor_map(&tmk4);
                prefetch_tensor_map(&tmv4);
            }
        }
    }
    __syncwarp();
    if (kClusters && nrank > 1) cluster_arrive();        // awaited before another CTA's memory is written: it has started
    // The suffix half starts while the prefix half runs.  That one began after every grid before it
    // had finished (it waits for them before it lets this one start), so queries, lengths, tables and
    // caches are in place; only its partial results are not, and the wait for those comes below.
    // (Loads here go past L1.  So every CTA of a prefix half, here and in pkv_prefill.cuh, waits before it triggers.)
    if constexpr (MODE == kSpanWindow || MODE == kSpanPrefix) pdl_wait();
    pdl_trigger();
    // (used once the lengths are here too: one round trip for all)
    const unsigned gave_up = *reinterpret_cast<const volatile unsigned int *>(&a.st->flags) & kFlagTimeout;

    // ---- this CTA's rows and tokens ----
    const int B = 1 << a.log2_block;
    const int item = blockIdx.x / nrank;
    const int tile = item % a.head_tiles, g = item / a.head_tiles % a.num_kv_heads, unit = item / a.head_tiles / a.num_kv_heads;
    int s = unit;                                       // whose table is read
    int first = 0, low = 0, ctx = 0, prefix = 0;        // visible: [0, first) and [low, ctx)
    int cols = min(a.tile_heads, a.group - tile * a.tile_heads);
    int row0 = unit * a.num_heads + g * a.group + tile * a.tile_heads;     // rows are numbered sequence * heads + head
    if constexpr (MODE == kSpanPrefix) {
        const int b = __ldcg(a.group_start + unit), e = __ldcg(a.group_start + unit + 1);
        const bool edge = (unit == 0 && b != 0) || (unit == a.num_groups - 1 && e != a.num_seqs);
        if (b < 0 || e < b || e > a.num_seqs || e - b > a.max_group || edge) {
            if (tid == 0 && g == 0 && tile == 0 && blockIdx.y == 0) latch(a.st, kFlagBadGroup, unit);
            if (b < 0 || e < b || e > a.num_seqs || e - b > a.max_group) return;
        }
        if (e == b) return;
        prefix = __ldcg(a.prefix_lens + b);
        const int most = min(a.max_prefix, __ldcg(a.ctx_lens + b));
        if (g == 0 && tile == 0 && blockIdx.y == 0)
            for (int i = b + tid; i < e; i += C::THREADS)
                if (__ldcg(a.prefix_lens + i) != prefix) latch(a.st, kFlagBadGroup, unit);
        // (one out of bounds is reported by the own tokens' half)
        if (prefix < 0 || prefix > most) return;
        low = blockIdx.y * a.parts.part;
        if (low >= prefix) return;
        ctx = min(prefix, low + a.parts.part);
        s = b;
        cols = min((e - b) * a.group - tile * COLS, COLS);
        if (cols <= 0) return;                                     // fewer rows than the largest group
        row0 = b * a.num_heads + g * a.group;
    } else {
        ctx = __ldcg(a.ctx_lens + s);
        if constexpr (MODE != kSpanWindow) prefix = __ldcg(a.prefix_lens + s);
        if (ctx < 0 || ctx > a.max_ctx) {
            if (tid == 0 && g == 0 && tile == 0 && rank == 0 && blockIdx.y == 0) latch(a.st, kFlagBadContext, ctx);
            ctx = ctx < 0 ? 0 : a.max_ctx;
        }
        if constexpr (MODE == kSpanWindow) {
            low = max(0, ctx - a.window);
            first = min(a.sinks, low);
        } else {
            if (prefix < 0 || prefix > ctx || prefix > a.max_prefix) {
                if (tid == 0 && g == 0 && tile == 0 && rank == 0 && blockIdx.y == 0) latch(a.st, kFlagBadContext, prefix);
                prefix = prefix < 0 ? 0 : min(ctx, a.max_prefix);
            }
            low = prefix;
            if constexpr (MODE == kSpanOwn) {           // this CTA's partition of them (the first one reports for all)
                low = (int)min((long long)ctx, prefix + (long long)blockIdx.y * a.parts.own);
                if (blockIdx.y + 1 < gridDim.y) ctx = low + min(ctx - low, a.parts.own);      // the last takes the rest
            }
        }
    }
    // row of column c (a group's columns run over its sequences, each with its heads of kv head g)
    auto row_of = [&](int c) -> size_t {
        if constexpr (MODE == kSpanPrefix) {
            const int r = tile * COLS + c;
            return (size_t)row0 + (size_t)(r / a.group) * a.num_heads + r % a.group;
        } else {
            return (size_t)row0 + c;
        }
    };
    // stages: those of the sinks, then those of [low, ctx); a stage that holds both counts once
    const int from = low / kTok;
    int nsink = (first + kTok - 1) / kTok;
    if (nsink > from) nsink = from;
    const int nst = low < ctx ? nsink + (ctx + kTok - 1) / kTok - from : 0;
    const int st0 = (int)((long long)nst * rank / nrank), st1 = (int)((long long)nst * (rank + 1) / nrank);
    bool dead = __any_sync(kFull, gave_up != 0);         // an earlier wait gave up: no copies, nothing waited for
    if (smem_u32(sm) & 1023u) {
        if (tid == 0) latch(a.st, kFlagTimeout, -2);
        dead = true;
    }
    const int mine = dead ? 0 : max(0, (st1 - st0 - warp + W - 1) / W);
    auto token0 = [&](int i) {                          // first token of this warp's stage i
        const int v = st0 + warp + W * i;
        return (v < nsink ? v : v - nsink + from) * kTok;
    };

    // ---- copies ----
    const int lcps = a.log2_block >= 4 ? 0 : 4 - a.log2_block;       // blocks per stage (log2)
    const int rows_per_copy = B < kTok ? B : kTok;
    const int per_load = 32 >> lcps;                                 // stages whose table entries one load brings
    const int32_t *table = a.tables + (size_t)s * a.max_blocks;
    auto seen_any = [&](int t, int n) { return t < ctx && (t < first || t + n > low); };       // of tokens t .. t + n - 1
    auto seen_all = [&](int t, int n) { return t + n <= ctx && (t >= low || t + n <= first); };
    auto load_entries = [&](int base) -> int {
        const int i = base + (lane >> lcps);
        if (i >= mine) return -1;
        const int t = token0(i) + (lane & ((1 << lcps) - 1)) * rows_per_copy;
        return seen_any(t, rows_per_copy) ? __ldcg(table + (t >> a.log2_block)) : -1;
    };
    const uint64_t policy = policy_evict_first();
    int ent = load_entries(0), base = 0;
    int ent_next = load_entries(per_load);
    // copy of this lane: half h of block j's keys (t = 0) or values (t = 1)
    const int ct = lane & 1, ch = (lane >> 1) % HALVES, cj = (lane >> 1) / HALVES;
    auto issue = [&](int i) {
        if (i == base + per_load) {
            base = i;
            ent = ent_next;
            ent_next = load_entries(base + per_load);
        }
        const int t0 = token0(i);
        const bool part = kFineBoxes && a.fine && !seen_all(t0, kTok);        // uniform over the warp
        const int rows = part ? kFine : rows_per_copy, off = cj * rows, t = t0 + off;
        const int p = __shfl_sync(kFull, ent, (((i - base) << lcps) + (lcps ? off >> a.log2_block : 0)) & 31);
        bool go = off < kTok && seen_any(t, rows);
        const bool bad = go && (p < 0 || p >= a.num_blocks);
        const unsigned badm = __ballot_sync(kFull, bad);
        if (badm) {
            if (lane == __ffs(badm) - 1) latch(a.st, kFlagBadBlock, p);
            go = go && !bad;
        }
        const unsigned n = __popc(__ballot_sync(kFull, go));
        const int slot = i % R;
        if (lane == 0) mbar_arrive_expect_tx(&full[slot], n * (uint32_t)rows * 128u);
        __syncwarp();
        if (go) {
            unsigned char *dst = ring + slot * C::STAGE_BYTES + ct * C::TENSOR_BYTES + ch * C::HALF_BYTES + off * 128;
            const void *map = part ? (ct ? &tmv4 : &tmk4) : (ct ? &tmv : &tmk);
            tma_load_4d(dst, map, ch * 64, t & (B - 1), g, p, &full[slot], policy);
        }
    };
    for (int i = 0; i < R && i < mine; i++) issue(i);

    // ---- queries: B fragments, column lane / 4 of each column tile, elements 2 (lane % 4) and + 8 of each step ----
    const int cq = lane & 3, r0 = lane >> 2;
    uint32_t qf[NT][D / 16][2];
#pragma unroll
    for (int n = 0; n < NT; n++) {
        const int c = 8 * n + r0;
        const bool there = c < cols && mine > 0;
        const uint32_t *qp = reinterpret_cast<const uint32_t *>(static_cast<const T *>(a.q) + (there ? row_of(c) : 0) * D) + cq;
#pragma unroll
        for (int k = 0; k < D / 16; k++) {
            qf[n][k][0] = there ? __ldcg(qp + 8 * k) : 0u;
            qf[n][k][1] = there ? __ldcg(qp + 8 * k + 4) : 0u;
        }
    }

    float o[NT][D / 16][4];                             // O^T: elements 16 i + r0 (+ 8), columns 2 cq, 2 cq + 1
    float m[NT][2], l[NT][2];
#pragma unroll
    for (int n = 0; n < NT; n++) {
#pragma unroll
        for (int i = 0; i < D / 16; i++)
#pragma unroll
            for (int e = 0; e < 4; e++) o[n][i][e] = 0.f;
        m[n][0] = m[n][1] = -INFINITY;
        l[n][0] = l[n][1] = 0.f;
    }

    // 16-byte chunk `chunk` of token row `row` in a tensor's stage (swizzled)
    auto chunk_at = [&](const unsigned char *t, int row, int chunk) {
        return t + (chunk >> 3) * C::HALF_BYTES + row * 128 + (((chunk & 7) ^ (row & 7)) << 4);
    };

    int i = 0;
    for (; i < mine; i++) {
        const int slot = i % R;
        if (!__all_sync(kFull, mbar_wait(&full[slot], (i / R) & 1, kWaitLimitCycles))) {
            if (lane == 0) latch(a.st, kFlagTimeout, i);
            dead = true;
            break;
        }
        const unsigned char *ks = ring + slot * C::STAGE_BYTES, *vs = ks + C::TENSOR_BYTES;
        const int t0 = token0(i);
        // S^T = K Q^T (even and odd steps apart: half the chain)
        float x[NT][4], y[NT][4];
#pragma unroll
        for (int n = 0; n < NT; n++)
#pragma unroll
            for (int e = 0; e < 4; e++) x[n][e] = y[n][e] = 0.f;
#pragma unroll
        for (int k = 0; k < D / 16; k += 2) {
            uint32_t f[4], h[4];
            ldmatrix_x4(f, chunk_at(ks, lane & 15, 2 * k + (lane >> 4)));
            ldmatrix_x4(h, chunk_at(ks, lane & 15, 2 * k + 2 + (lane >> 4)));
#pragma unroll
            for (int n = 0; n < NT; n++) {
                Mma<T>::run(x[n], f, qf[n][k][0], qf[n][k][1]);
                Mma<T>::run(y[n], h, qf[n][k + 1][0], qf[n][k + 1][1]);
            }
        }
#pragma unroll
        for (int n = 0; n < NT; n++)
#pragma unroll
            for (int e = 0; e < 4; e++) x[n][e] = (x[n][e] + y[n][e]) * a.scale_log2;
        // tokens of the stage that the rows see (the same for every row)
        const bool whole = seen_all(t0, kTok);
        uint32_t vm0 = ~0u, vm1 = ~0u;                  // value fragments: tokens 2 cq, 2 cq + 1, and those + 8
        if (!whole) {
            auto seen = [&](int t) { return t0 + t < ctx && (t0 + t >= low || t0 + t < first); };
            if (!seen(r0)) {
#pragma unroll
                for (int n = 0; n < NT; n++) x[n][0] = x[n][1] = -INFINITY;
            }
            if (!seen(r0 + 8)) {
#pragma unroll
                for (int n = 0; n < NT; n++) x[n][2] = x[n][3] = -INFINITY;
            }
            vm0 = (seen(2 * cq) ? 0xffffu : 0u) | (seen(2 * cq + 1) ? 0xffff0000u : 0u);
            vm1 = (seen(2 * cq + 8) ? 0xffffu : 0u) | (seen(2 * cq + 9) ? 0xffff0000u : 0u);
        }
        // running maximum and sum; P^T as the second product's B operand
        uint32_t ph[NT][2], pl[NT][2];
#pragma unroll
        for (int n = 0; n < NT; n++) {
            float m0 = fmaxf(x[n][0], x[n][2]), m1 = fmaxf(x[n][1], x[n][3]);
#pragma unroll
            for (int d = 4; d <= 16; d <<= 1) {
                m0 = fmaxf(m0, __shfl_xor_sync(kFull, m0, d));
                m1 = fmaxf(m1, __shfl_xor_sync(kFull, m1, d));
            }
            if (__any_sync(kFull, m0 > m[n][0] || m1 > m[n][1])) {
                m0 = fmaxf(m[n][0], m0);
                m1 = fmaxf(m[n][1], m1);
                const float a0 = m0 == -INFINITY ? 1.f : ex2(m[n][0] - m0), a1 = m1 == -INFINITY ? 1.f : ex2(m[n][1] - m1);
                m[n][0] = m0;
                m[n][1] = m1;
                l[n][0] *= a0;
                l[n][1] *= a1;
#pragma unroll
                for (int j = 0; j < D / 16; j++) {
                    o[n][j][0] *= a0;
                    o[n][j][1] *= a1;
                    o[n][j][2] *= a0;
                    o[n][j][3] *= a1;
                }
            }
            const float z0 = m[n][0] == -INFINITY ? 0.f : m[n][0], z1 = m[n][1] == -INFINITY ? 0.f : m[n][1];
            const float p0 = ex2(x[n][0] - z0), p1 = ex2(x[n][1] - z1), p2 = ex2(x[n][2] - z0), p3 = ex2(x[n][3] - z1);
            l[n][0] += p0 + p2;
            l[n][1] += p1 + p3;
            uint32_t hi0, lo0, hi1, lo1;
            split_pair<T>(p0, p1, hi0, lo0);
            split_pair<T>(p2, p3, hi1, lo1);
            ph[n][0] = movmatrix_trans(hi0);
            ph[n][1] = movmatrix_trans(hi1);
            pl[n][0] = movmatrix_trans(lo0);
            pl[n][1] = movmatrix_trans(lo1);
        }
        // O^T += V^T P^T
#pragma unroll
        for (int j = 0; j < D / 16; j++) {
            uint32_t f[4];
            ldmatrix_x4_trans(f, chunk_at(vs, (lane & 7) + ((lane >> 4) << 3), 2 * j + ((lane >> 3) & 1)));
            if (!whole) {
                f[0] &= vm0;
                f[1] &= vm0;
                f[2] &= vm1;
                f[3] &= vm1;
            }
#pragma unroll
            for (int n = 0; n < NT; n++) {
                Mma<T>::run(o[n][j], f, ph[n][0], ph[n][1]);
                Mma<T>::run(o[n][j], f, pl[n][0], pl[n][1]);
            }
        }
        __syncwarp();                                   // the slot has been read
        if (i + R < mine) issue(i + R);
    }
    if (dead)                                           // copies in flight land before their memory is reused
        for (int k = i; k < min(i + R, mine); k++) mbar_wait(&full[k % R], (k / R) & 1, kDrainLimitCycles);
    __syncwarp();

    // ---- the warps' parts, through their rings ----
    float *wo = reinterpret_cast<float *>(ring);
    float *wml = reinterpret_cast<float *>(sm + C::wml) + warp * 2 * COLS;
#pragma unroll
    for (int n = 0; n < NT; n++) {
#pragma unroll
        for (int d = 4; d <= 16; d <<= 1) {
            l[n][0] += __shfl_xor_sync(kFull, l[n][0], d);
            l[n][1] += __shfl_xor_sync(kFull, l[n][1], d);
        }
        const int c = 8 * n + 2 * cq;
        if (r0 == 0) {
            wml[c] = m[n][0];
            wml[c + 1] = m[n][1];
            wml[COLS + c] = l[n][0];
            wml[COLS + c + 1] = l[n][1];
        }
#pragma unroll
        for (int j = 0; j < D / 16; j++) {
            wo[c * LD + 16 * j + r0] = o[n][j][0];
            wo[(c + 1) * LD + 16 * j + r0] = o[n][j][1];
            wo[c * LD + 16 * j + r0 + 8] = o[n][j][2];
            wo[(c + 1) * LD + 16 * j + r0 + 8] = o[n][j][3];
        }
    }
    __syncthreads();
    const float *all_ml = reinterpret_cast<const float *>(sm + C::wml);
    auto join_warps = [&](int c, int e) {
        Joined r{-INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
#pragma unroll
        for (int w = 0; w < W; w++)
            r.add(all_ml[w * 2 * COLS + c], all_ml[w * 2 * COLS + COLS + c],
                  *reinterpret_cast<const float4 *>(sm + w * C::ring_bytes + (c * LD + e) * 4));
        return r;
    };
    constexpr int UPR = D / 4;                          // units of four elements per row
    auto store_out = [&](int c, int e, const Joined &r) {
        const float inv = r.l > 0.f ? 1.f / r.l : 0.f;
        uint2 w;
        w.x = Mma<T>::pack(r.o.x * inv, r.o.y * inv);
        w.y = Mma<T>::pack(r.o.z * inv, r.o.w * inv);
        *reinterpret_cast<uint2 *>(static_cast<T *>(a.out) + row_of(c) * D + e) = w;
    };
    auto store_part = [&](int c, int e, const Joined &r) {
        const size_t at = row_of(c) * a.parts.slots + (MODE == kSpanPrefix ? 0 : a.parts.max_parts) + blockIdx.y;
        *reinterpret_cast<float4 *>(a.parts.o + at * D + e) = r.o;
        if (e == 0) {
            a.parts.m[at] = r.m;
            a.parts.l[at] = r.l;
        }
    };
    if constexpr (MODE == kSpanPrefix || MODE == kSpanOwn) {
        if (nst > 0)
            for (int u = tid; u < cols * UPR; u += C::THREADS) {
                const int c = u / UPR, e = u % UPR * 4;
                store_part(c, e, join_warps(c, e));
            }
        // what follows the own tokens' grid waits for it alone: it may not end before the prefix half
        if constexpr (MODE == kSpanOwn)
            if (blockIdx.x == gridDim.x - 1 && blockIdx.y == gridDim.y - 1) pdl_wait();
    } else {
        const int np = MODE == kSpanSuffix ? (prefix + a.parts.part - 1) / a.parts.part : 0;
        auto join_prefix = [&](int c, int e, Joined &r) {
            const size_t at = row_of(c) * a.parts.slots;
            for (int p0 = 0; p0 < np; p0 += 4) {                    // four parts to a round trip
                float pm[4], pl2[4];
                float4 po[4];
#pragma unroll
                for (int p = 0; p < 4; p++) {
                    const bool there = p0 + p < np;
                    pm[p] = there ? __ldcg(a.parts.m + at + p0 + p) : -INFINITY;
                    pl2[p] = there ? __ldcg(a.parts.l + at + p0 + p) : 0.f;
                    po[p] = there ? __ldcg(reinterpret_cast<const float4 *>(a.parts.o + (at + p0 + p) * D + e))
                                  : make_float4(0.f, 0.f, 0.f, 0.f);
                }
#pragma unroll
                for (int p = 0; p < 4; p++) r.add(pm[p], pl2[p], po[p]);
            }
        };
        if (!kClusters || nrank == 1) {
            if constexpr (MODE == kSpanSuffix) pdl_wait();          // the prefix half's results
            for (int u = tid; u < cols * UPR; u += C::THREADS) {
                const int c = u / UPR, e = u % UPR * 4;
                Joined r = join_warps(c, e);
                if constexpr (MODE == kSpanSuffix) join_prefix(c, e, r);
                store_out(c, e, r);
            }
        } else if constexpr (kClusters) {
            // CTA k of the cluster joins the units k, k + nrank, ...: every CTA writes its part of them into
            // that CTA's shared memory, so that after one barrier each reads its own
            const int share = (cols * UPR + (int)nrank - 1) / (int)nrank;
            __syncwarp();
            cluster_wait();
            const uint32_t got = smem_u32(sm + C::got), got_ml = smem_u32(sm + C::got_ml);
            for (int u = tid; u < cols * UPR; u += C::THREADS) {
                const Joined r = join_warps(u / UPR, u % UPR * 4);
                const uint32_t to = (uint32_t)u % nrank, at = rank * (uint32_t)share + (uint32_t)u / nrank;
                st_cluster4(map_rank(got + at * 16, to), r.o);
                st_cluster2(map_rank(got_ml + at * 8, to), r.m, r.l);
            }
            __syncwarp();
            cluster_arrive();
            if constexpr (MODE == kSpanSuffix) pdl_wait();
            cluster_wait();
            const float4 *go = reinterpret_cast<const float4 *>(sm + C::got);
            const float2 *gm = reinterpret_cast<const float2 *>(sm + C::got_ml);
            for (int i = tid, u; (u = i * (int)nrank + (int)rank) < cols * UPR; i += C::THREADS) {
                const int c = u / UPR, e = u % UPR * 4;
                float M = -INFINITY;
                for (uint32_t k = 0; k < nrank; k++) M = fmaxf(M, gm[k * share + i].x);
                const float z = M == -INFINITY ? 0.f : M;
                Joined r{M, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
#pragma unroll 4
                for (uint32_t k = 0; k < nrank; k++) {
                    const float2 ml = gm[k * share + i];
                    const float4 v = go[k * share + i];
                    const float w = ex2(ml.x - z);
                    r.l = fmaf(ml.y, w, r.l);
                    r.o.x = fmaf(v.x, w, r.o.x);
                    r.o.y = fmaf(v.y, w, r.o.y);
                    r.o.z = fmaf(v.z, w, r.o.z);
                    r.o.w = fmaf(v.w, w, r.o.w);
                }
                if constexpr (MODE == kSpanSuffix) join_prefix(c, e, r);
                store_out(c, e, r);
            }
        }
    }
}

// Joins a row's parts, those of its prefix and of its own tokens: a warp per row,
// four parts to a round trip.
constexpr int kJoinWarps = 8;

template <int D, typename T>
__global__ void __launch_bounds__(kJoinWarps * 32)
    span_join_kernel(T *out, const int32_t *ctx_lens, const int32_t *prefix_lens, int rows, int num_heads, int max_ctx,
                     int max_prefix, PrefixParts parts) {
    constexpr int E = D / 32;
    pdl_wait();
    pdl_trigger();
    const int row = blockIdx.x * kJoinWarps + threadIdx.x / 32, lane = threadIdx.x & 31;
    if (row >= rows) return;
    const int s = row / num_heads;
    const int ctx = min(max(__ldcg(ctx_lens + s), 0), max_ctx), prefix = min(max(__ldcg(prefix_lens + s), 0), min(ctx, max_prefix));
    const int np = (prefix + parts.part - 1) / parts.part;
    const int n = np + min((ctx - prefix + parts.own - 1) / parts.own, parts.slots - parts.max_parts);
    const int skip = parts.max_parts - np;                                       // own parts come last
    const size_t at = (size_t)row * parts.slots;
    float M = -INFINITY, L = 0.f, o[E];
#pragma unroll
    for (int e = 0; e < E; e++) o[e] = 0.f;
    for (int p0 = 0; p0 < n; p0 += 4) {
        float pm[4], pl[4], po[4][E];
#pragma unroll
        for (int p = 0; p < 4; p++) {
            const bool there = p0 + p < n;
            const size_t k = at + p0 + p + (p0 + p < np ? 0 : skip);
            pm[p] = there ? __ldcg(parts.m + k) : -INFINITY;
            pl[p] = there ? __ldcg(parts.l + k) : 0.f;
#pragma unroll
            for (int e = 0; e < E; e += 2) {
                const float2 v = there ? __ldcg(reinterpret_cast<const float2 *>(parts.o + k * D + lane * E + e))
                                       : make_float2(0.f, 0.f);
                po[p][e] = v.x;
                po[p][e + 1] = v.y;
            }
        }
        float Mn = M;
#pragma unroll
        for (int p = 0; p < 4; p++) Mn = fmaxf(Mn, pm[p]);
        const float z = Mn == -INFINITY ? 0.f : Mn, a = ex2(M - z);
        M = Mn;
        L *= a;
#pragma unroll
        for (int e = 0; e < E; e++) o[e] *= a;
#pragma unroll
        for (int p = 0; p < 4; p++) {
            const float w = ex2(pm[p] - z);
            L = fmaf(pl[p], w, L);
#pragma unroll
            for (int e = 0; e < E; e++) o[e] = fmaf(po[p][e], w, o[e]);
        }
    }
    const float inv = L > 0.f ? 1.f / L : 0.f;
    uint32_t *dst = reinterpret_cast<uint32_t *>(out + (size_t)row * D + lane * E);
#pragma unroll
    for (int e = 0; e < E; e += 2) dst[e / 2] = Mma<T>::pack(o[e] * inv, o[e + 1] * inv);
}

// The cache [NB][Hkv][B][D] as a 4-D tensor (innermost first); a box is 64
// elements of d by min(B, tokens) tokens of one (block, kv head).
bool encode_span_map(CUtensorMap *map, const void *base, int num_blocks, int Hkv, int B, int D, bool bf16, int tokens) {
    const cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)B, (cuuint64_t)Hkv, (cuuint64_t)(num_blocks > 0 ? num_blocks : 1)};
    const cuuint64_t strides[3] = {(cuuint64_t)D * 2, (cuuint64_t)B * D * 2, (cuuint64_t)Hkv * B * D * 2};
    const cuuint32_t box[4] = {64u, (cuuint32_t)(B < tokens ? B : tokens), 1u, 1u};
    return encode_tiled16(map, base, 4, dims, strides, box, bf16);
}

struct SpanMaps {
    CUtensorMap k, v, k4, v4;
};

template <int D, int NT, int W, typename T, int MODE>
cudaError_t launch_span_kernel(const SpanArgs &a, const SpanMaps &maps, long long items, int parts, int cluster, cudaStream_t st) {
    auto kern = span_attention_kernel<D, NT, W, T, MODE>;
    using C = SpanConf<D, NT, W>;
    static std::atomic<unsigned long long> sized{0}, wide{0};
    cudaError_t e = allow_smem(kern, C::bytes, sized);
    if (e != cudaSuccess) return e;
    if (cluster > 8) {                                   // more than the portable size, once per device
        int d = 0;
        if ((e = cudaGetDevice(&d)) != cudaSuccess) return e;
        const unsigned long long bit = d < 64 ? 1ull << d : 0ull;
        if (!(wide.load(std::memory_order_acquire) & bit)) {
            e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
            if (e != cudaSuccess) return e;
            wide.fetch_or(bit, std::memory_order_release);
        }
    }
    return launch_clusters(kern, dim3((unsigned)(items * cluster), (unsigned)parts), dim3(C::THREADS), (unsigned)cluster,
                           C::bytes, st, a, maps.k, maps.v, maps.k4, maps.v4);
}

// How a launch is spread: warps per CTA, CTAs per cluster.
struct Spread {
    int warps, cluster;
};

// (prefixes go by CTAs of four warps, own tokens in partitions by CTAs of two; the others by either)
template <int D, int NT, typename T, int MODE>
cudaError_t launch_span_warps(const SpanArgs &a, const SpanMaps &maps, long long items, int parts, Spread w, cudaStream_t st) {
    if constexpr (MODE != kSpanPrefix)
        if (MODE == kSpanOwn || w.warps == 2) return launch_span_kernel<D, NT, 2, T, MODE>(a, maps, items, parts, 1, st);
    if constexpr (MODE != kSpanOwn) return launch_span_kernel<D, NT, 4, T, MODE>(a, maps, items, parts, w.cluster, st);
}

template <int MODE>
cudaError_t launch_span(int D, int NT, bool bf16, const SpanArgs &a, const SpanMaps &maps, long long items, int parts,
                        Spread w, cudaStream_t st) {
    using B = __nv_bfloat16;
    using F = __half;
    if (D == 128 && NT == 1)
        return bf16 ? launch_span_warps<128, 1, B, MODE>(a, maps, items, parts, w, st)
                    : launch_span_warps<128, 1, F, MODE>(a, maps, items, parts, w, st);
    if (D == 128)
        return bf16 ? launch_span_warps<128, 2, B, MODE>(a, maps, items, parts, w, st)
                    : launch_span_warps<128, 2, F, MODE>(a, maps, items, parts, w, st);
    if (NT == 1)
        return bf16 ? launch_span_warps<64, 1, B, MODE>(a, maps, items, parts, w, st)
                    : launch_span_warps<64, 1, F, MODE>(a, maps, items, parts, w, st);
    return bf16 ? launch_span_warps<64, 2, B, MODE>(a, maps, items, parts, w, st)
                : launch_span_warps<64, 2, F, MODE>(a, maps, items, parts, w, st);
}

// Work items (sequence, kv head) of up to max_tokens tokens over the GPU.  CTAs are
// of two warps where those of four would come in a second, nearly empty wave or
// the items are short and many (each item's start and end then weighs more than
// its stream): 512 items of 512 tokens 25.1 against 30.6 us, of 2,048 tokens 83 against
// 97, 8,192 of 64 tokens 59 against 74; but 2,048 of 1,024 tokens 163 against 157.
// Clusters split items while they leave SMs without one, or with one and long
// streams: 8 items of 4,096 tokens 27, 15.8, 10.8, 9.7 us for 2, 4, 8, 16 CTAs each
// (8.6 for 16 since their parts are written and not read across the cluster);
// 128 of 512 tokens 10.1 us unsplit, 10.9 in two.  (head_dim 128, bf16.)
Spread choose_spread(long long items, long long max_tokens, int NT) {
    const long long sms = sm_count(), four = sms * (NT == 1 ? 3 : 2);      // CTAs of four warps that fit at once
    const long long stages = (max_tokens + kTok - 1) / kTok;
    if (items > four) return {items <= 2 * four || stages <= 32 ? 2 : 4, 1};
    int c = 1;
    while (c < kMaxCluster && items * c * 2 <= 2 * sms && stages >= (items * c * 2 <= sms ? 16 : 32) * c * 2) c *= 2;
    if (c == 1 && stages >= 128) c = 2;                  // few and long: the SMs' shares differ by less
    return {4, c};
}

struct SpanCall {
    const char *what;
    const void *out, *query, *key_cache, *value_cache;
    const int32_t *block_tables, *context_lens;
    int num_seqs, max_blocks, max_context_len, block_size, num_blocks, num_heads, num_kv_heads, head_dim;
    float scale;
    pkv_dtype dtype;
};

// The checks that both calls share; fills what the kernels need of the arguments.
pkv_status check_span(const SpanCall &c, SpanArgs &a) {
    if (c.dtype != PKV_F16 && c.dtype != PKV_BF16) return fail(PKV_EINVAL, "%s: bad dtype %d", c.what, (int)c.dtype);
    if (c.num_seqs < 0 || c.num_seqs > 65535 || c.max_blocks < 0 || c.num_blocks < 0)
        return fail(PKV_EINVAL, "%s: bad sizes (seqs %d, table width %d, blocks %d)", c.what, c.num_seqs, c.max_blocks,
                    c.num_blocks);
    if (c.head_dim != 64 && c.head_dim != 128)
        return fail(PKV_EINVAL, "%s: head_dim %d not supported (64 or 128)", c.what, c.head_dim);
    if (!is_pow2(c.block_size) || c.block_size < 4 || c.block_size > 128)
        return fail(PKV_EINVAL, "%s: block_size %d not a power of two in [4, 128]", c.what, c.block_size);
    if (c.num_heads <= 0 || c.num_kv_heads <= 0 || c.num_heads % c.num_kv_heads || c.num_heads > 65535)
        return fail(PKV_EINVAL, "%s: %d query heads do not group over %d kv heads (at most 65535)", c.what, c.num_heads,
                    c.num_kv_heads);
    if ((long long)c.num_seqs * c.num_heads > 1 << 30)
        return fail(PKV_EINVAL, "%s: %d sequences of %d query heads (at most 2^30 rows)", c.what, c.num_seqs, c.num_heads);
    if (!std::isfinite(c.scale)) return fail(PKV_EINVAL, "%s: scale must be finite", c.what);
    const int64_t cap = (int64_t)c.max_blocks * c.block_size;
    if (c.max_context_len < 0 || c.max_context_len > cap)
        return fail(PKV_EINVAL, "%s: max_context_len %d beyond the table (%lld tokens)", c.what, c.max_context_len,
                    (long long)cap);
    const int64_t most = c.max_context_len > 0 ? c.max_context_len : cap;
    if (most > (1 << 30)) return fail(PKV_EINVAL, "%s: contexts of more than 2^30 tokens", c.what);
    if (c.num_seqs == 0) return PKV_OK;
    if (!c.out || !c.query || !c.key_cache || !c.value_cache || !c.block_tables || !c.context_lens)
        return fail(PKV_EINVAL, "%s: NULL pointer", c.what);
    if (!aligned16(c.out) || !aligned16(c.query) || !aligned16(c.key_cache) || !aligned16(c.value_cache))
        return fail(PKV_EINVAL, "%s: pointers must be 16-byte aligned", c.what);
    a.out = const_cast<void *>(c.out);
    a.q = c.query;
    a.tables = c.block_tables;
    a.ctx_lens = c.context_lens;
    a.num_seqs = c.num_seqs;
    a.max_blocks = c.max_blocks;
    a.max_ctx = (int)most;
    a.log2_block = ilog2(c.block_size);
    a.num_blocks = c.num_blocks;
    a.num_heads = c.num_heads;
    a.num_kv_heads = c.num_kv_heads;
    a.group = c.num_heads / c.num_kv_heads;
    a.head_tiles = (a.group + 15) / 16;
    a.tile_heads = (a.group + a.head_tiles - 1) / a.head_tiles;
    a.scale_log2 = (float)((double)c.scale * 1.4426950408889634);
    return PKV_OK;
}

// What a checked call needs of the device.
pkv_status open_span(const SpanCall &c, SpanArgs &a, SpanMaps &maps) {
    a.st = status_ptr();
    if (!a.st) return fail(PKV_ECUDA, "%s: no device status word", c.what);
    const bool bf16 = c.dtype == PKV_BF16;
    std::memset(&maps, 0, sizeof maps);
    auto encode = [&](CUtensorMap *map, const void *cache, int tokens) {
        return encode_span_map(map, cache, c.num_blocks, c.num_kv_heads, c.block_size, c.head_dim, bf16, tokens);
    };
    // Items beyond one wave are bound by memory: at head_dim 128 they read the edges of what is seen in
    // boxes of four tokens (a window of 64 and 4 sinks are 6 stages, 96 tokens, as a rule; so 72).  8,192
    // items with windows of 64, 128, 256, 1,024: 58.4, 94.7, 165.4, 492 us without, 53.6, 85.8, 154.7, 483
    // with.  At head_dim 64 it is slower (window 128: 55.6 against 58.5 us: the small copies count for more);
    // fewer items wait for round trips, and the two maps more would only cost their callers.
    const long long items = (long long)c.num_seqs * c.num_kv_heads * a.head_tiles;
    a.fine = c.head_dim == 128 && c.block_size > kFine && items > 3ll * sm_count();
    if (!encode(&maps.k, c.key_cache, kTok) || !encode(&maps.v, c.value_cache, kTok) ||
        (a.fine && (!encode(&maps.k4, c.key_cache, kFine) || !encode(&maps.v4, c.value_cache, kFine))))
        return fail(PKV_ECUDA, "%s: no tensor map of the cache", c.what);
    return PKV_OK;
}

// ---- sequences that share a prefix -------------------------------------------

// A column tile of the kernel above holds this many query rows per kv head
// (sequences x heads).  Larger groups take several, each with its own pass over the
// prefix, while the passes of the call come to no more than this many tokens and kv
// heads; the rest goes to the tcgen05 kernel, whose start costs some 5 us more.  (8
// sequences of 32/8 heads after 1,024 tokens 8.3 against 11.5 us, after 8,192 18.4
// against 18.3; 64 after 512 14.5 against 15.0, after 2,048 31 against 18.)
constexpr int kFewRows = 16;
constexpr long long kFewPasses = 1 << 16;

// How a call is split.
struct SharedPlan {
    bool few;                    // the prefixes go through the kernel above
    int part, max_parts;         // tokens of a prefix's partition (a multiple of 128), partitions
    int own, own_parts;          // of a sequence's own tokens, where the join is a launch of its own
    int prefix_ctas;             // SMs for the prefixes, where own tokens run beside them
    size_t m_off, l_off, o_off, bytes;
};

SharedPlan plan_shared(int S, int groups, int H, int Hkv, int D, int max_prefix, int max_group, int max_suffix) {
    SharedPlan w{};
    const int group = H / Hkv, tiles = (max_prefix + 127) / 128;
    const int sms = sm_count() > 0 ? sm_count() : 152;   // (a size asked for where there is no GPU)
    const long long col_tiles = ((long long)max_group * group + kFewRows - 1) / kFewRows;
    w.few = col_tiles == 1 || col_tiles * groups * Hkv * std::max(1, max_prefix) <= kFewPasses;
    int per = tiles > 0 ? tiles : 1;                     // key tiles of a partition
    if (w.few) {
        // CTAs in waves; a key tile's time in us at full occupancy, or when the GPU is not full, a CTA's
        // start and end, the parts' way through L2 (16 groups of 8 after 1,024 tokens, 32 heads: one
        // partition leaves a second wave of 56 CTAs: 72 us in all, 68 with four)
        const long long units = (long long)groups * Hkv * col_tiles, slots = sms * ((long long)max_group * group > 8 ? 2 : 3);
        const double full = 128 * 4.0 * D / (6.6e6 / slots);
        double least = 1e300;
        for (int p = 1, last = 0; p <= tiles && p <= 64; p++) {
            const int tp = (tiles + p - 1) / p;
            if (tp == last) continue;
            last = tp;
            const int parts = (tiles + tp - 1) / tp;
            const long long ctas = units * parts, waves = (ctas + slots - 1) / slots;
            const double tile = full * std::max(0.7, std::min(1.0, (double)ctas / slots));
            const double cost = waves * (tp * tile + 3.0) + (double)parts * S * H * D * 8.0 / 8e6;
            if (cost < least) {
                least = cost;
                per = tp;
            }
        }
    } else {
        // The prefixes are bound by the tensor cores and run on n SMs; own tokens are bound by memory
        // and run on the others, then on all.  Times in us, measured on the kernels: a key tile of 256
        // rows 2.0, of 128 or fewer 1.4 (between fp16's and bf16's), an item's start and end 6; an SM
        // reads up to 85 KB/us, all of them 6.6 MB/us; parts pass through L2 at 8 MB/us.
        const int seqs = 2 * (128 / group);
        const double t = (long long)S * group > 128ll * groups ? 2.0 : 1.4;
        const long long units = std::max<long long>(groups, (S + seqs - 1) / seqs) * Hkv;
        const double token = 4.0 * Hkv * D, prefix_bytes = token * groups * max_prefix, own_bytes = token * S * max_suffix / 2;
        double least = 1e300;
        int last = 0;
        for (int p = 1; p <= tiles && p <= 64; p++) {
            const int tp = (tiles + p - 1) / p;
            if (tp == last) continue;
            last = tp;
            const int parts = (tiles + tp - 1) / tp;
            const long long items = units * parts;
            for (long long k = (items + sms - 1) / sms, end = k + 3; k <= end; k++) {
                const int n = (int)((items + k - 1) / k);
                const double t_prefix = (double)((items + n - 1) / n) * (tp * t + 6.0);
                const double beside = std::max(0.0, std::min(6.6e6 - prefix_bytes / t_prefix, (sms - n) * 85e3));
                const double cost = t_prefix + std::max(0.0, own_bytes - beside * t_prefix) / 6.6e6 +
                                    (double)parts * S * H * D * 8.0 / 8e6;
                if (cost < least) {
                    least = cost;
                    per = tp;
                    w.prefix_ctas = n;
                }
            }
        }
        if (w.prefix_ctas < 1) w.prefix_ctas = 1;
        // own tokens in partitions of about 512, at most 16 (128 requests of up to 1,024 own tokens after
        // 8,190 shared ones: 61 us; partitions of 256 64, of 128 70)
        w.own_parts = std::min(16, std::max(1, (max_suffix + 511) / 512));
        w.own = std::max(kTok, ((max_suffix + w.own_parts - 1) / w.own_parts + kTok - 1) / kTok * kTok);
    }
    w.part = per * 128;
    w.max_parts = tiles > per ? (tiles + per - 1) / per : 1;      // (one where no prefix is: its launch is always made)
    const size_t n = (size_t)S * H * (w.max_parts + w.own_parts);
    w.l_off = align256(n * sizeof(float));
    w.o_off = w.l_off + align256(n * sizeof(float));
    w.bytes = w.o_off + align256(n * D * sizeof(float));
    return w;
}

template <int D, typename T> cudaError_t launch_join(const SpanArgs &a, cudaStream_t st) {
    const int rows = a.num_seqs * a.num_heads;
    return launch(span_join_kernel<D, T>, dim3((unsigned)((rows + kJoinWarps - 1) / kJoinWarps)), dim3(kJoinWarps * 32), 0, st,
                  static_cast<T *>(a.out), a.ctx_lens, a.prefix_lens, rows, a.num_heads, a.max_ctx, a.max_prefix, a.parts);
}

}  // namespace
}  // namespace pkv

extern "C" {

pkv_status paged_attention_decode_window(void *out, const void *query, const void *key_cache, const void *value_cache,
                                         const int32_t *block_tables, const int32_t *context_lens, int num_seqs,
                                         int max_blocks_per_seq, int max_context_len, int block_size, int num_blocks,
                                         int num_heads, int num_kv_heads, int head_dim, float scale, int window,
                                         int num_sinks, pkv_dtype dtype, struct CUstream_st *stream) {
    using namespace pkv;
    const char *what = "paged_attention_decode_window";
    if (window < 1 || num_sinks < 0)
        return fail(PKV_EINVAL, "%s: window %d (at least 1), %d sinks (at least 0)", what, window, num_sinks);
    const SpanCall call = {what, out, query, key_cache, value_cache, block_tables, context_lens, num_seqs,
                           max_blocks_per_seq, max_context_len, block_size, num_blocks, num_heads, num_kv_heads, head_dim,
                           scale, dtype};
    SpanArgs a = {};
    SpanMaps maps;
    pkv_status rc = check_span(call, a);
    if (rc != PKV_OK || num_seqs == 0) return rc;
    rc = open_span(call, a, maps);
    if (rc != PKV_OK) return rc;
    a.window = window;
    a.sinks = num_sinks;
    const int NT = a.tile_heads > 8 ? 2 : 1;
    const long long items = (long long)num_seqs * num_kv_heads * a.head_tiles;
    const long long tokens = std::min<long long>(a.max_ctx, (long long)window + num_sinks);
    const cudaError_t e = launch_span<kSpanWindow>(head_dim, NT, dtype == PKV_BF16, a, maps, items, 1,
                                                   choose_spread(items, tokens, NT), stream);
    if (e != cudaSuccess) return fail(PKV_ECUDA, "%s: launch: %s", what, cudaGetErrorString(e));
    return PKV_OK;
}

size_t paged_attention_decode_shared_workspace_size(int num_seqs, int num_groups, int num_heads, int num_kv_heads,
                                                    int head_dim, int max_context_len, int max_prefix_len,
                                                    int max_group_size, int max_suffix_len) {
    using namespace pkv;
    if (num_seqs <= 0 || num_groups <= 0 || num_heads <= 0 || num_kv_heads <= 0 || num_heads % num_kv_heads ||
        num_heads / num_kv_heads > 128 || head_dim <= 0 || max_context_len < 0 || max_prefix_len < 0 || max_group_size < 0 ||
        max_suffix_len < 0)
        return 0;
    if (max_group_size == 0 || max_group_size > num_seqs) max_group_size = num_seqs;
    if (max_prefix_len == 0 || max_prefix_len > max_context_len) max_prefix_len = max_context_len;
    if (max_suffix_len == 0 || max_suffix_len > max_context_len) max_suffix_len = max_context_len;
    return plan_shared(num_seqs, num_groups, num_heads, num_kv_heads, head_dim, max_prefix_len, max_group_size,
                       max_suffix_len).bytes;
}

pkv_status paged_attention_decode_shared(void *out, const void *query, const void *key_cache, const void *value_cache,
                                         const int32_t *block_tables, const int32_t *context_lens,
                                         const int32_t *group_start, const int32_t *prefix_lens, int num_seqs,
                                         int num_groups, int max_group_size, int max_prefix_len, int max_suffix_len,
                                         int max_blocks_per_seq, int max_context_len, int block_size, int num_blocks,
                                         int num_heads, int num_kv_heads, int head_dim, float scale, void *workspace,
                                         size_t workspace_bytes, pkv_dtype dtype, struct CUstream_st *stream) {
    using namespace pkv;
    const char *what = "paged_attention_decode_shared";
    if (num_groups < 0 || max_group_size < 0 || max_prefix_len < 0 || max_suffix_len < 0)
        return fail(PKV_EINVAL, "%s: negative size (groups %d, largest group %d, prefix %d, suffix %d)", what, num_groups,
                    max_group_size, max_prefix_len, max_suffix_len);
    if (num_groups > num_seqs && num_seqs >= 0)
        return fail(PKV_EINVAL, "%s: %d groups of %d sequences", what, num_groups, num_seqs);
    if (!(scale > 0.f)) return fail(PKV_EINVAL, "%s: scale must be positive", what);
    const SpanCall call = {what, out, query, key_cache, value_cache, block_tables, context_lens, num_seqs,
                           max_blocks_per_seq, max_context_len, block_size, num_blocks, num_heads, num_kv_heads, head_dim,
                           scale, dtype};
    SpanArgs a = {};
    SpanMaps maps;
    pkv_status rc = check_span(call, a);
    if (rc != PKV_OK || num_seqs == 0) return rc;
    if (num_groups == 0) return fail(PKV_EINVAL, "%s: no groups", what);
    if (!group_start || !prefix_lens) return fail(PKV_EINVAL, "%s: NULL pointer", what);
    if (a.group > 128) return fail(PKV_EINVAL, "%s: %d query heads per kv head (at most 128)", what, a.group);
    if (max_prefix_len > a.max_ctx)
        return fail(PKV_EINVAL, "%s: max_prefix_len %d beyond the contexts (%d tokens)", what, max_prefix_len, a.max_ctx);
    const int max_prefix = max_prefix_len > 0 ? max_prefix_len : a.max_ctx;
    const int max_group = max_group_size == 0 || max_group_size > num_seqs ? num_seqs : max_group_size;
    a.prefix_lens = prefix_lens;
    a.group_start = group_start;
    a.num_groups = num_groups;
    a.max_prefix = max_prefix;
    a.max_group = max_group;
    const bool bf16 = dtype == PKV_BF16;
    const int max_suffix = max_suffix_len > 0 && max_suffix_len < a.max_ctx ? max_suffix_len : a.max_ctx;
    cudaError_t e = cudaSuccess;
    const SharedPlan w = plan_shared(num_seqs, num_groups, num_heads, num_kv_heads, head_dim, max_prefix, max_group,
                                     max_suffix);
    if (!workspace || workspace_bytes < w.bytes || !aligned16(workspace))
        return fail(PKV_EINVAL, "%s: workspace of %zu bytes needed, %zu given", what, w.bytes,
                    workspace ? workspace_bytes : (size_t)0);
    const long long prefix_items = ((long long)num_groups + more_pairs(num_seqs, max_group, a.group)) * w.max_parts * num_kv_heads;
    if (!w.few && prefix_items > kMaxSharedItems)
        return fail(PKV_EINVAL, "%s: %lld work items ((groups + further pairs of row tiles) x partitions x kv heads) above 2^27",
                    what, prefix_items);
    rc = open_span(call, a, maps);
    if (rc != PKV_OK) return rc;
    unsigned char *ws = static_cast<unsigned char *>(workspace);
    a.parts = {reinterpret_cast<float *>(ws + w.m_off), reinterpret_cast<float *>(ws + w.l_off),
               reinterpret_cast<float *>(ws + w.o_off), w.part, w.max_parts, w.own, w.max_parts + w.own_parts};
    const int NT = a.tile_heads > 8 ? 2 : 1;
    const long long items = (long long)num_seqs * num_kv_heads * a.head_tiles;
    if (w.few) {
        // the prefixes, then the sequences' own tokens and the join
        const long long rows = (long long)max_group * a.group;
        SpanArgs p = a;
        p.head_tiles = (int)((rows + kFewRows - 1) / kFewRows);
        p.fine = 0;
        e = launch_span<kSpanPrefix>(head_dim, rows > 8 ? 2 : 1, bf16, p, maps,
                                     (long long)num_groups * num_kv_heads * p.head_tiles, w.max_parts, {4, 1}, stream);
        if (e == cudaSuccess) e = launch_span<kSpanSuffix>(head_dim, NT, bf16, a, maps, items, 1,
                                                          choose_spread(items, max_suffix, NT), stream);
    } else {
        // the prefixes on some of the SMs, own tokens beside them on the others, then the join
        e = launch_shared_prefix(query, key_cache, value_cache, block_tables, context_lens, group_start, prefix_lens, num_groups, num_seqs,
                                 max_group, max_prefix, max_blocks_per_seq, block_size, num_blocks, num_heads,
                                 num_kv_heads, head_dim, a.scale_log2, a.parts, bf16, w.prefix_ctas, stream);
        if (e == cudaSuccess)
            e = launch_span<kSpanOwn>(head_dim, NT, bf16, a, maps, items, w.own_parts, {2, 1}, stream);
        if (e == cudaSuccess)
            e = head_dim == 128 ? bf16 ? launch_join<128, __nv_bfloat16>(a, stream) : launch_join<128, __half>(a, stream)
                : bf16          ? launch_join<64, __nv_bfloat16>(a, stream)
                                : launch_join<64, __half>(a, stream);
    }
    if (e != cudaSuccess) return fail(PKV_ECUDA, "%s: launch: %s", what, cudaGetErrorString(e));
    return PKV_OK;
}

}  // extern "C"
