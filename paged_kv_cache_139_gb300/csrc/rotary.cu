// Rotary positions on the way into the paged cache.
//
// Pair i of a head's first `rotary_dim` elements, (x[i], x[i + r/2]) in the
// half layout or (x[2i], x[2i + 1]) in the interleaved one, is turned by the
// angle p * theta_i of its token's position p:
//     (a, b) -> (a cos - b sin, a sin + b cos),  theta_i = base^(-2i / r),
// the other elements pass through.  The cosines and sines come from a table
// [positions][r / 2][2] that rotary_table writes once per program.
//
// The append kernels rotate the queries into query_out and the keys into the
// cache, and copy the values, in one launch: each element is read once and
// written once, which is what bounds them.
#include <cfloat>
#include <cmath>
#include <cstring>

#include "pkv_fp8.cuh"
#include "pkv_host.cuh"

namespace pkv {
namespace {

constexpr int kMaxRotaryDim = 256;
constexpr int kMaxPositions = 1 << 30;      // of a table: positions and strides past its end stay in 31 bits
constexpr int kRopeThreads = 256;

// ---- the table ---------------------------------------------------------------

// theta_i / 2 pi as a 64-bit fraction of a turn: position p's angle is
// p * turn mod 2^64, exact whatever p, with no 64-bit floating point on the
// device (the low bits of a far position's angle are all that 32-bit
// arithmetic would keep).
struct TurnTable {
    unsigned long long turn[kMaxRotaryDim / 2];
};

// Cosines and sines of two 64-bit fractions of a turn, (cos, sin, cos, sin): the
// nearest quarter turn swaps and negates; what is left, y within pi / 4 of zero,
// takes the Taylor series of both (to y^9 and y^10: the next terms are below
// 2^-29 and 2^-33), the two angles in one instruction each.
__device__ __forceinline__ float4 cos_sin_of(unsigned long long turns0, unsigned long long turns1, float magnitude) {
    const unsigned t0 = (unsigned)(turns0 >> 32), t1 = (unsigned)(turns1 >> 32);    // fractions of a turn, 2^-32 units
    const unsigned q0 = (t0 + 0x20000000u) >> 30, q1 = (t1 + 0x20000000u) >> 30;    // nearest quarter turns
    const auto both = [](float x) { return pack2(x, x); };
    const unsigned long long y = mul2(pack2((float)(int)(t0 - (q0 << 30)), (float)(int)(t1 - (q1 << 30))),
                                      both(1.4629180792671596e-9f));                // 2 pi / 2^32
    const unsigned long long z = mul2(y, y);
    unsigned long long s = fma2(z, both(1.f / 362880.f), both(-1.f / 5040.f));
    s = fma2(z, s, both(1.f / 120.f));
    s = fma2(z, s, both(-1.f / 6.f));
    s = fma2(mul2(y, z), s, y);
    unsigned long long c = fma2(z, both(-1.f / 3628800.f), both(1.f / 40320.f));
    c = fma2(z, c, both(-1.f / 720.f));
    c = fma2(z, c, both(1.f / 24.f));
    c = fma2(z, c, both(-0.5f));
    c = fma2(z, c, both(1.f));
    s = mul2(s, both(magnitude));
    c = mul2(c, both(magnitude));
    // quarter turns 1 and 3 swap; the cosine changes its sign in 1 and 2, the sine in 2 and 3
    const float c0 = (q0 & 1) ? lo2(s) : lo2(c), s0 = (q0 & 1) ? lo2(c) : lo2(s);
    const float c1 = (q1 & 1) ? hi2(s) : hi2(c), s1 = (q1 & 1) ? hi2(c) : hi2(s);
    const auto flip = [](float x, unsigned q) { return __uint_as_float(__float_as_uint(x) ^ ((q & 2u) << 30)); };
    return make_float4(flip(c0, q0 + 1u), flip(s0, q0), flip(c1, q1 + 1u), flip(s1, q1));
}

// Thread t owns two neighbouring pairs (one 16-byte store) of every
// (threads / columns)-th position of its CTA's stretch: its turns stay in
// registers.  131,072 x 128: 11.2 us, 6.0 TB/s written.
__global__ void __launch_bounds__(kRopeThreads) rotary_table_kernel(float4 *__restrict__ out,
                                                                    const __grid_constant__ TurnTable tab,
                                                                    int num_positions, int columns, int rows,
                                                                    int per_cta, float magnitude) {
    pdl_trigger();
    pdl_wait();
    const int c = threadIdx.x % columns, r = threadIdx.x / columns;
    if (r >= rows) return;
    const unsigned long long t0 = tab.turn[2 * c], t1 = tab.turn[2 * c + 1];
    const int begin = blockIdx.x * per_cta;
    const int end = begin + per_cta < num_positions ? begin + per_cta : num_positions;
    for (int p = begin + r; p < end; p += rows) {
        out[(size_t)p * columns + c] =
            cos_sin_of(t0 * (unsigned long long)p, t1 * (unsigned long long)p, magnitude);
    }
}

// ---- rotating sixteen elements --------------------------------------------------

struct RopeArgs {
    const void *q, *k, *v;         // [T][H or Hkv][D], tokens q_stride / k_stride / v_stride elements apart
    void *q_out;                   // [T][H][D]
    void *k_cache, *v_cache;       // [NB][Hkv][B][D]
    float *scales;                 // 8-bit cache: [NB][scale_heads][2]
    const float *cos_sin;          // [num_positions][rot / 2][2]
    const int32_t *positions;      // [T]
    const int64_t *slots;          // [T]
    DeviceStatus *st;
    int64_t q_stride, k_stride, v_stride;
    int64_t num_slots;
    int num_tokens, num_heads, num_kv_heads;
    int rot, num_positions, log2_block;
    // 8-bit append: see rotary_append8_kernel
    int single_ctas, single_tokens, single_parts;
    int run_ctas, run_tokens, group_heads;
    unsigned long long run_share;  // 2^32 times the share of run_ctas in the CTAs that they are mixed into
};

// A thread's unit of a head: sixteen elements as two 16-byte chunks that
// begin at elements a and b.  Unit u below rot / 16 holds pairs 8u .. 8u + 7
// whole, in either layout; the units after it hold what is not rotated.
struct Unit {
    int a, b;
    bool rotated;
};

template <bool INTERLEAVED> __device__ __forceinline__ Unit unit_at(int u, int rot) {
    Unit x;
    x.rotated = u * 16 < rot;
    const bool half = !INTERLEAVED && x.rotated;
    x.a = half ? 8 * u : 16 * u;
    x.b = half ? rot / 2 + 8 * u : 16 * u + 8;
    return x;
}

// The eight (cos, sin) of unit u at position p.
__device__ __forceinline__ void load_cos_sin(float4 (&cs)[4], const RopeArgs &a, int p, int u) {
    const float4 *t = reinterpret_cast<const float4 *>(a.cos_sin + (size_t)p * a.rot + u * 16);
#pragma unroll
    for (int i = 0; i < 4; i++) cs[i] = __ldg(t + i);
}

// x[0..7] = chunk a, x[8..15] = chunk b, turned in place.  The products and
// their sum are rounded one by one (no fused multiply-add), so that the
// result is that of the formula in 32 bits, whoever evaluates it: a value on
// the border between two 8-bit codes then falls the same way.  (Instructions
// on two numbers at once do not serve: the assembler fuses their products and
// sums.)
template <bool INTERLEAVED> __device__ __forceinline__ void turn(float (&x)[16], const float4 (&cs)[4]) {
#pragma unroll
    for (int i = 0; i < 8; i++) {
        const float c = (i & 1) ? cs[i >> 1].z : cs[i >> 1].x;
        const float s = (i & 1) ? cs[i >> 1].w : cs[i >> 1].y;
        const int ia = INTERLEAVED ? 2 * i : i, ib = INTERLEAVED ? 2 * i + 1 : i + 8;
        const float u = x[ia], v = x[ib];
        x[ia] = __fsub_rn(__fmul_rn(u, c), __fmul_rn(v, s));
        x[ib] = __fadd_rn(__fmul_rn(u, s), __fmul_rn(v, c));
    }
}

template <typename T> __device__ __forceinline__ void widen(float (&x)[16], const uint4 &ra, const uint4 &rb) {
    float f[8];
    F16Traits<T>::to_f32(ra, f);
#pragma unroll
    for (int i = 0; i < 8; i++) x[i] = f[i];
    F16Traits<T>::to_f32(rb, f);
#pragma unroll
    for (int i = 0; i < 8; i++) x[8 + i] = f[i];
}

template <typename T> __device__ __forceinline__ uint4 narrow(const float *x) {
    return make_uint4(Mma<T>::pack(x[0], x[1]), Mma<T>::pack(x[2], x[3]), Mma<T>::pack(x[4], x[5]),
                      Mma<T>::pack(x[6], x[7]));
}

// A token's position, or -1 outside the table (latched by the thread that
// tells, but for padding tokens).
__device__ __forceinline__ int checked_position(const RopeArgs &a, int t, bool tell) {
    const int p = a.positions[t];
    if (p >= 0 && p < a.num_positions) return p;
    if (tell && a.slots[t] >= 0) latch(a.st, kFlagBadPosition, p);
    return -1;
}

// Rotates unit u of one row of a 16-bit tensor into another.
template <typename T, bool INTERLEAVED>
__device__ __forceinline__ void rotate_row(const RopeArgs &a, const T *src, T *dst, int u, int pos) {
    const Unit x = unit_at<INTERLEAVED>(u, a.rot);
    uint4 ra = *reinterpret_cast<const uint4 *>(src + x.a);
    uint4 rb = *reinterpret_cast<const uint4 *>(src + x.b);
    if (x.rotated) {
        float4 cs[4];
        load_cos_sin(cs, a, pos, u);
        float f[16];
        widen<T>(f, ra, rb);
        turn<INTERLEAVED>(f, cs);
        ra = narrow<T>(f);
        rb = narrow<T>(f + 8);
    }
    *reinterpret_cast<uint4 *>(dst + x.a) = ra;
    *reinterpret_cast<uint4 *>(dst + x.b) = rb;
}

// ---- append to the 16-bit cache ---------------------------------------------------

// One thread per unit of a row; the rows of a token are its query heads, its
// key heads and its value heads.  16,381 tokens of 32/8 heads: 62.4 us, 6.5 TB/s,
// the rate of a copy; 256 tokens of 32/32 heads: 4.3 us in a captured graph.
template <int D, typename T, bool INTERLEAVED>
__global__ void __launch_bounds__(kRopeThreads) rotary_append_kernel(const RopeArgs a) {
    constexpr int UPR = D / 16;
    pdl_trigger();
    pdl_wait();
    const unsigned per_token = (unsigned)(a.num_heads + 2 * a.num_kv_heads) * UPR;
    const unsigned long long i = (unsigned long long)blockIdx.x * kRopeThreads + threadIdx.x;
    const unsigned long long t64 = i / per_token;
    if (t64 >= (unsigned)a.num_tokens) return;
    const int t = (int)t64;
    const int r = (int)(i - t64 * per_token);
    int row = r / UPR;
    const int u = r % UPR;
    if (row < a.num_heads) {
        const int pos = checked_position(a, t, r == 0);
        if (pos < 0) return;
        rotate_row<T, INTERLEAVED>(a, static_cast<const T *>(a.q) + t * a.q_stride + row * D,
                                   static_cast<T *>(a.q_out) + ((size_t)t * a.num_heads + row) * D, u, pos);
        return;
    }
    row -= a.num_heads;
    const bool isv = row >= a.num_kv_heads;
    const int h = isv ? row - a.num_kv_heads : row;
    const int64_t s = a.slots[t];
    if (s < 0) return;                                     // padding token
    const int pos = checked_position(a, t, row == 0 && u == 0 && a.num_heads == 0);
    if (s >= a.num_slots) {
        if (row == 0 && u == 0) latch(a.st, kFlagBadSlot, s);
        return;
    }
    if (pos < 0) return;
    const int64_t blk = s >> a.log2_block, off = s & ((1ll << a.log2_block) - 1);
    const size_t dst = (size_t)(((blk * a.num_kv_heads + h) << a.log2_block) + off) * D;
    if (isv) {
        const uint4 *src = reinterpret_cast<const uint4 *>(static_cast<const T *>(a.v) + t * a.v_stride + h * D) + 2 * u;
        uint4 *out = reinterpret_cast<uint4 *>(static_cast<T *>(a.v_cache) + dst) + 2 * u;
        const uint4 x = src[0], y = src[1];
        out[0] = x;
        out[1] = y;
    } else {
        rotate_row<T, INTERLEAVED>(a, static_cast<const T *>(a.k) + t * a.k_stride + h * D,
                                   static_cast<T *>(a.k_cache) + dst, u, pos);
    }
}

// ---- append to the 8-bit cache ----------------------------------------------------

// Neighbouring tokens of the call that go to one block: n of them from token t.
struct Run {
    int t, n;
    bool fresh;                // one of them is the block's first row
};

// The run that begins at token t (whose slot is in block blk), by the whole warp.
__device__ __forceinline__ Run find_run(const RopeArgs &a, int t, int64_t blk, int lane) {
    Run run;
    run.t = t;
    run.n = 0;
    run.fresh = false;
    for (int base = t; base < a.num_tokens; base += 32) {
        const int i = base + lane;
        const int64_t s = i < a.num_tokens ? __ldg(a.slots + i) : -1;
        const bool in = s >= 0 && s < a.num_slots && (s >> a.log2_block) == blk;
        const unsigned m = __ballot_sync(0xffffffffu, in);
        const int cnt = m == 0xffffffffu ? 32 : __ffs(~m) - 1;
        run.fresh |= __any_sync(0xffffffffu, lane < cnt && (s & ((1ll << a.log2_block) - 1)) == 0);
        run.n += cnt;
        if (cnt < 32) break;
    }
    return run;
}

// The run's offsets in its block as bits (block sizes up to 128), by the whole warp.
struct Rows {
    unsigned bits[4];
};

__device__ __forceinline__ Rows written_rows(const RopeArgs &a, const Run &run, int lane) {
    Rows w;
    w.bits[0] = w.bits[1] = w.bits[2] = w.bits[3] = 0u;
    for (int base = 0; base < run.n; base += 32) {
        const bool in = base + lane < run.n;
        const int off = in ? (int)(__ldg(a.slots + run.t + base + lane) & ((1ll << a.log2_block) - 1)) : 0;
#pragma unroll
        for (int k = 0; k < 4; k++)
            w.bits[k] |= __reduce_or_sync(0xffffffffu, in && (off >> 5) == k ? 1u << (off & 31) : 0u);
    }
    return w;
}

__device__ __forceinline__ bool was_written(const Rows &w, int off) {
    const unsigned b = off < 64 ? (off < 32 ? w.bits[0] : w.bits[1]) : (off < 96 ? w.bits[2] : w.bits[3]);
    return (b >> (off & 31)) & 1u;
}

// Whether slot x is in the pool and in slot s's block.
__device__ __forceinline__ bool same_block(const RopeArgs &a, int64_t x, int64_t s) {
    return x >= 0 && x < a.num_slots && (x >> a.log2_block) == (s >> a.log2_block);
}

__device__ __forceinline__ float *scale_of(const RopeArgs &a, int64_t blk, int h, bool isv) {
    return a.scales + ((size_t)blk * scale_heads(a.num_kv_heads) + h) * 2 + (isv ? 1 : 0);
}

// Sixteen codes under a scale 1 / ratio times as large.
__device__ __forceinline__ void round_again(uint4 *q, float ratio) {
    const uint4 w = *q;
    const uint32_t in[4] = {w.x, w.y, w.z, w.w};
    uint32_t out[4];
#pragma unroll
    for (int j = 0; j < 4; j++) {
        const uint32_t lo = e4m3x2_lo(in[j]), hi = e4m3x2_hi(in[j]);
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&lo));
        const float2 g = __half22float2(*reinterpret_cast<const __half2 *>(&hi));
        out[j] = to_e4m3x4(f.x * ratio, f.y * ratio, g.x * ratio, g.y * ratio);
    }
    *q = make_uint4(out[0], out[1], out[2], out[3]);
}

// The block's scale for new rows of magnitude up to amax, stored;
// the block's other rows are rounded again where it grows.  `had`: the scale
// before, not looked at when the run starts the block anew.  By one warp.
template <int D>
__device__ __forceinline__ float grow_scale(const RopeArgs &a, const Run &run, float *sp, float had, float amax,
                                            unsigned char *rows, int lane) {
    constexpr int UPR = D / 16, RP = 32 / UPR;
    const int r = lane / UPR, u = lane % UPR;
    amax = fminf(amax, 3.4028235e38f);             // infinities; NaN does not come this far
    // a write at offset 0 starts the block anew; otherwise its scale can only grow
    if (run.fresh) had = 0.f;
    const float scale = fmaxf(had, pow2_scale(amax));
    if (!run.fresh && scale != had) {
        const Rows written = written_rows(a, run, lane);
        const float ratio = __fdiv_rn(had, scale);
        for (int o = r; o < 1 << a.log2_block; o += RP) {
            if (was_written(written, o)) continue;
            round_again(reinterpret_cast<uint4 *>(rows + (size_t)o * D) + u, ratio);
        }
    }
    __syncwarp();
    if (lane == 0) *sp = scale;
    return scale;
}

// A unit's codes under `scale` into its row.  The reciprocal of a power of two
// is exact; a caller's own scale may be another number.
__device__ __forceinline__ void store_codes(unsigned char *row, const Unit &x, float (&f)[16], float scale) {
    if ((__float_as_uint(scale) & 0x7fffffu) == 0u && scale < 0x1p126f) {
        const float inv = __uint_as_float(0x7f000000u - __float_as_uint(scale));   // 2^-e
#pragma unroll
        for (int e = 0; e < 16; e += 2) {
            const unsigned long long y = mul2(pack2(f[e], f[e + 1]), pack2(inv, inv));
            f[e] = lo2(y);
            f[e + 1] = hi2(y);
        }
    } else {
#pragma unroll
        for (int e = 0; e < 16; e++) f[e] = __fdiv_rn(f[e], scale);
    }
    *reinterpret_cast<uint2 *>(row + x.a) =
        make_uint2(to_e4m3x4(f[0], f[1], f[2], f[3]), to_e4m3x4(f[4], f[5], f[6], f[7]));
    *reinterpret_cast<uint2 *>(row + x.b) =
        make_uint2(to_e4m3x4(f[8], f[9], f[10], f[11]), to_e4m3x4(f[12], f[13], f[14], f[15]));
}

// A run of one token, the usual one of a decode step: its key and value rows j
// = j0 + lane / (D/16) (the keys of `heads` kv heads from h0 on, then their
// values) side by side.
template <int D, typename T, bool INTERLEAVED>
__device__ __forceinline__ void append8_token(const RopeArgs &a, int t, int pos, int64_t slot, bool fresh, int h0,
                                              int heads, int j0, int lane) {
    constexpr int UPR = D / 16;
    const int u = lane % UPR, j = j0 + lane / UPR;
    const bool active = j < 2 * heads, isv = j >= heads;
    const int h = h0 + (isv ? j - heads : j);
    const int off = (int)(slot & ((1ll << a.log2_block) - 1));
    const int64_t blk = slot >> a.log2_block;
    const Unit x = unit_at<INTERLEAVED>(u, isv ? 0 : a.rot);
    float y[16];
    float amax = 0.f, had = 0.f;
    if (active) {
        const T *src = isv ? static_cast<const T *>(a.v) + t * a.v_stride + h * D
                           : static_cast<const T *>(a.k) + t * a.k_stride + h * D;
        const uint4 ra = *reinterpret_cast<const uint4 *>(src + x.a), rb = *reinterpret_cast<const uint4 *>(src + x.b);
        if (!fresh) had = *scale_of(a, blk, h, isv);
        widen<T>(y, ra, rb);
        if (x.rotated && pos >= 0 && pos < a.num_positions) {
            float4 cs[4];
            load_cos_sin(cs, a, pos, u);
            turn<INTERLEAVED>(y, cs);
        }
#pragma unroll
        for (int e = 0; e < 16; e++) amax = fmaxf(amax, fabsf(y[e]));
    }
#pragma unroll
    for (int o = UPR / 2; o >= 1; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    if (!active) return;
    const float scale = fmaxf(had, pow2_scale(fminf(amax, 3.4028235e38f)));
    unsigned char *rows = static_cast<unsigned char *>(isv ? a.v_cache : a.k_cache) +
                          ((size_t)(blk * a.num_kv_heads + h) << a.log2_block) * D;
    if (!fresh && scale != had) {
        const float ratio = __fdiv_rn(had, scale);
#pragma unroll 4
        for (int o = 0; o < 1 << a.log2_block; o++)
            if (o != off) round_again(reinterpret_cast<uint4 *>(rows + (size_t)o * D) + u, ratio);
    }
    if (u == 0) *scale_of(a, blk, h, isv) = scale;
    store_codes(rows + (size_t)off * D, x, y, scale);
}

// The largest magnitude of eight 16-bit values, NaN passed over (zero if all are NaN: a
// NaN's bits would win the maximum that is taken over bits after this).
template <typename T> __device__ __forceinline__ float largest8(const uint4 &w);
template <> __device__ __forceinline__ float largest8<__half>(const uint4 &w) {
    const __half2 *h = reinterpret_cast<const __half2 *>(&w);
    const __half2 m = __hmax2(__hmax2(__habs2(h[0]), __habs2(h[1])), __hmax2(__habs2(h[2]), __habs2(h[3])));
    return fmaxf(0.f, fmaxf(__low2float(m), __high2float(m)));
}
template <> __device__ __forceinline__ float largest8<__nv_bfloat16>(const uint4 &w) {
    const __nv_bfloat162 *h = reinterpret_cast<const __nv_bfloat162 *>(&w);
    const __nv_bfloat162 m = __hmax2(__hmax2(__habs2(h[0]), __habs2(h[1])), __hmax2(__habs2(h[2]), __habs2(h[3])));
    return fmaxf(0.f, fmaxf(__low2float(m), __high2float(m)));
}

// Sixteen bytes of shared memory in one load (the compiler would split it by
// the elements that it feeds, at four times the bank accesses).
__device__ __forceinline__ uint4 load_shared16(const void *p) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(smem_u32(p)));
    return v;
}

// CTAs of three kinds.
//  * Runs of one token (a decode step's): a CTA looks over single_tokens tokens
//    for them, a warp to key and value rows of one side by side; in small calls
//    single_parts CTAs share a token's heads.  Bound by latency: everything
//    that a token needs is requested as soon as its slot is known.
//  * Longer runs (prompts): a CTA looks over run_tokens tokens for those that
//    begin a run (about one of block_size does) and takes group_heads kv heads of
//    it.  The run's keys and values come as bulk copies of whole row pieces into
//    shared memory, 32 KB at a time with five CTAs to an SM, which keeps more
//    bytes under way than registers hold.  A thread keeps to one unit of a row,
//    whose cosines it holds, and goes through the heads' keys and values twice:
//    for the magnitudes, and, when the scales are known, for the codes.
//  * Queries: a thread to a unit of four heads.  These wait for memory while the
//    second kind computes, so the two are mixed in the grid (16,381 tokens of
//    32/32 heads: 124 us with the queries last, 114 so; of 32/8: 68 and 59).
// 16,381 tokens of 32/32 heads: 114 us, 6.0 TB/s (200 with two passes of loads
// into registers, 133 with 64 KB and 256 threads to a CTA, half on keys and half
// on values); a step of 256 tokens of 32/8 heads: 2.8 us in a captured graph.
constexpr int kAppend8Threads = 128;
constexpr int kAppend8Ctas = 5;                                     // to an SM
constexpr int kSlabBytes = 32 * 1024;                               // one head of a block of 128 takes twice that
constexpr int kMaxGroupHeads = kSlabBytes / (4 * 64 * 4);           // blocks of 4 tokens, head_dim 64
constexpr int kQueryRows = 4;
static_assert(2 * kMaxGroupHeads <= kAppend8Threads, "a thread clears a magnitude");

template <int D, typename T, bool INTERLEAVED>
__global__ void __launch_bounds__(kAppend8Threads, kAppend8Ctas) rotary_append8_kernel(const RopeArgs a) {
    constexpr int UPR = D / 16;
    constexpr int W = kAppend8Threads / 32;
    extern __shared__ __align__(16) unsigned char slab[];           // [2][rows][group_heads][D] 16-bit
    __shared__ uint64_t bar;
    __shared__ int failed;
    __shared__ unsigned top[2 * kMaxGroupHeads];                    // largest magnitudes, then scales, as bits
    if (threadIdx.x == 0) {
        mbar_init(&bar, 1);
        fence_mbar_init();
        failed = 0;
    }
    __syncthreads();                       // any warp may issue the first copies
    pdl_trigger();
    pdl_wait();
    if (blockIdx.x < (unsigned)a.single_ctas) {
        const int lane = threadIdx.x & 31, part = (int)blockIdx.x % a.single_parts;
        const int base = (int)blockIdx.x / a.single_parts * a.single_tokens;
        const int around = base - 1 + lane;                           // the window and a token to either side
        const int64_t s = lane < a.single_tokens + 2 && around >= 0 && around < a.num_tokens ? __ldg(a.slots + around) : -1;
        const int p = a.rot && around >= 0 && around < a.num_tokens ? __ldg(a.positions + around) : -1;
        const int64_t before = __shfl_up_sync(0xffffffffu, s, 1), after = __shfl_down_sync(0xffffffffu, s, 1);
        const bool alone = lane >= 1 && lane <= a.single_tokens && s >= 0 && s < a.num_slots &&
                           !same_block(a, before, s) && !same_block(a, after, s);
        const int jobs = (2 * a.num_kv_heads + 32 / UPR - 1) / (32 / UPR);
        int done = 0;                                                 // jobs of the tokens before
        for (unsigned todo = __ballot_sync(0xffffffffu, alone); todo; todo &= todo - 1, done += jobs) {
            const int l = __ffs(todo) - 1;
            const int64_t slot = __shfl_sync(0xffffffffu, s, l);
            const int pos = __shfl_sync(0xffffffffu, p, l);
            for (int j = part * W + ((int)(threadIdx.x >> 5) + W - done % W) % W; j < jobs; j += a.single_parts * W)
                append8_token<D, T, INTERLEAVED>(a, base - 1 + l, pos, slot, (slot & ((1ll << a.log2_block) - 1)) == 0,
                                                 0, a.num_kv_heads, j * (32 / UPR), lane);
        }
        return;
    }
    // this CTA's number among those that append runs, or those that rotate queries
    const unsigned cta = blockIdx.x - a.single_ctas;
    const int runs_before = min((int)((cta * a.run_share) >> 32), a.run_ctas);
    if (runs_before == a.run_ctas || (int)(((cta + 1) * a.run_share) >> 32) == runs_before) {
        const unsigned groups = (unsigned)(a.num_heads + kQueryRows - 1) / kQueryRows;
        const unsigned per_token = groups * UPR;
        const unsigned long long i = (unsigned long long)(cta - runs_before) * kAppend8Threads + threadIdx.x;
        const unsigned long long t64 = i / per_token;
        if (t64 >= (unsigned)a.num_tokens) return;
        const int t = (int)t64;
        const int r = (int)(i - t64 * per_token);
        const int row0 = (r / UPR) * kQueryRows, u = r % UPR;
        const int n = a.num_heads - row0 < kQueryRows ? a.num_heads - row0 : kQueryRows;
        const Unit x = unit_at<INTERLEAVED>(u, a.rot);
        const T *src = static_cast<const T *>(a.q) + t * a.q_stride + row0 * D;
        T *dst = static_cast<T *>(a.q_out) + ((size_t)t * a.num_heads + row0) * D;
        uint4 ra[kQueryRows], rb[kQueryRows];
#pragma unroll
        for (int k = 0; k < kQueryRows; k++)
            if (k < n) {
                ra[k] = *reinterpret_cast<const uint4 *>(src + k * D + x.a);
                rb[k] = *reinterpret_cast<const uint4 *>(src + k * D + x.b);
            }
        const int pos = checked_position(a, t, r == 0);
        if (pos < 0) return;
        float4 cs[4];
        if (x.rotated) load_cos_sin(cs, a, pos, u);
#pragma unroll
        for (int k = 0; k < kQueryRows; k++)
            if (k < n) {
                if (x.rotated) {
                    float f[16];
                    widen<T>(f, ra[k], rb[k]);
                    turn<INTERLEAVED>(f, cs);
                    ra[k] = narrow<T>(f);
                    rb[k] = narrow<T>(f + 8);
                }
                *reinterpret_cast<uint4 *>(dst + k * D + x.a) = ra[k];
                *reinterpret_cast<uint4 *>(dst + k * D + x.b) = rb[k];
            }
        return;
    }
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int B = 1 << a.log2_block;
    const int hgroups = (a.num_kv_heads + a.group_heads - 1) / a.group_heads;
    const int h0 = (runs_before % hgroups) * a.group_heads;
    const int heads = a.num_kv_heads - h0 < a.group_heads ? a.num_kv_heads - h0 : a.group_heads;
    const int first = (runs_before / hgroups) * a.run_tokens;
    const int last = first + a.run_tokens < a.num_tokens ? first + a.run_tokens : a.num_tokens;
    const uint32_t piece = (uint32_t)(heads * D * sizeof(T));        // of a token's row
    // this thread's unit, its row of rows_at_once (whole warps of them), and its first head of every head_step-th
    const int rows_at_once = min(max(B, 32 / UPR), kAppend8Threads / UPR), head_step = kAppend8Threads / UPR / rows_at_once;
    const int r = tid / UPR % rows_at_once, u = tid % UPR, head0 = tid / UPR / rows_at_once;
    const Unit xk = unit_at<INTERLEAVED>(u, a.rot), xv = unit_at<INTERLEAVED>(u, 0);
    if (tid == 0 && timed_out(a.st)) failed = 1;
    uint32_t phase = 0;
    for (int base = first; base < last; base += 32) {
        // the tokens that begin a run, a lane to a token; every warp finds the same ones
        const int tl = base + lane;
        const bool mine = tl < last;
        const int64_t sl = mine ? __ldg(a.slots + tl) : -1;
        const int64_t before = mine && tl > 0 ? __ldg(a.slots + tl - 1) : -1;
        const int64_t after = mine && tl + 1 < a.num_tokens ? __ldg(a.slots + tl + 1) : -1;
        const bool good = sl >= 0 && sl < a.num_slots;
        if (h0 == 0 && warp == 0 && sl >= 0) {
            if (a.rot) checked_position(a, tl, a.num_heads == 0);
            if (!good) latch(a.st, kFlagBadSlot, sl);
        }
        // but for runs of one token: other CTAs take them
        const bool leads = good && !same_block(a, before, sl) && same_block(a, after, sl);
        for (unsigned todo = __ballot_sync(0xffffffffu, leads); todo; todo &= todo - 1) {
            const int src_lane = __ffs(todo) - 1, t = base + src_lane;
            const int64_t blk = __shfl_sync(0xffffffffu, sl, src_lane) >> a.log2_block;
            Run run = find_run(a, t, blk, lane);
            if (run.n > B) run.n = B;                                 // slots that repeat: the slab holds a block
            if (tid < 2 * heads) top[tid] = 0;
            if (tid == 0) mbar_arrive_expect_tx(&bar, 2u * (uint32_t)run.n * piece);
            // row pieces of keys, then of values, spread over the warps
            for (int c = lane * W + warp; c < 2 * run.n; c += kAppend8Threads) {
                const bool v = c >= run.n;
                const int row = v ? c - run.n : c;
                const T *src = v ? static_cast<const T *>(a.v) + (t + row) * a.v_stride
                                 : static_cast<const T *>(a.k) + (t + row) * a.k_stride;
                bulk_g2s(slab + (size_t)c * piece, src + (size_t)h0 * D, piece, &bar);
            }
            // meanwhile this thread's first row: its offset in the block and its cosines
            int off = 0;
            bool turned = false;
            float4 cs[4];
            auto plan = [&](int row) {
                turned = false;
                if (row >= run.n) return;
                off = (int)(__ldg(a.slots + t + row) & (B - 1));
                if (xk.rotated) {
                    const int pos = __ldg(a.positions + t + row);
                    turned = pos >= 0 && pos < a.num_positions;       // others have been latched
                    if (turned) load_cos_sin(cs, a, pos, u);
                }
            };
            plan(r);
            if (!mbar_wait(&bar, phase, kWaitLimitCycles)) {
                if (lane == 0) latch(a.st, kFlagTimeout, t);
                failed = 1;
            }
            __syncthreads();
            if (failed) {                                             // copies may still be under way
                if (tid == 0) mbar_wait(&bar, phase, kDrainLimitCycles);
                return;
            }
            phase ^= 1u;
            const T *keys = reinterpret_cast<const T *>(slab), *values = keys + (size_t)run.n * heads * D;
            auto key32 = [&](float (&y)[16], int row, int h) {
                const T *q = keys + (row * heads + h) * D;
                widen<T>(y, load_shared16(q + xk.a), load_shared16(q + xk.b));
                if (turned) turn<INTERLEAVED>(y, cs);
            };
            for (int row0 = 0; row0 < run.n; row0 += rows_at_once) {
                const int row = row0 + r;
                if (row0 > 0) plan(row);
                for (int h = head0; h < heads; h += head_step) {
                    float kmax = 0.f, vmax = 0.f;
                    if (row < run.n) {
                        const T *q = values + (row * heads + h) * D;
                        vmax = fmaxf(largest8<T>(load_shared16(q + xv.a)), largest8<T>(load_shared16(q + xv.b)));
                        if (turned) {
                            float y[16];
                            key32(y, row, h);
#pragma unroll
                            for (int e = 0; e < 16; e++) kmax = fmaxf(kmax, fabsf(y[e]));
                        } else {
                            q = keys + (row * heads + h) * D;
                            kmax = fmaxf(largest8<T>(load_shared16(q + xk.a)), largest8<T>(load_shared16(q + xk.b)));
                        }
                    }
                    // magnitudes are not negative: their bits order as they do
                    const unsigned km = __reduce_max_sync(0xffffffffu, __float_as_uint(kmax));
                    const unsigned vm = __reduce_max_sync(0xffffffffu, __float_as_uint(vmax));
                    if (lane < 2) atomicMax(&top[2 * h + lane], lane ? vm : km);
                }
            }
            __syncthreads();
            for (int j = warp; j < 2 * heads; j += W) {
                const bool v = j & 1;
                const int h = h0 + (j >> 1);
                unsigned char *rows = static_cast<unsigned char *>(v ? a.v_cache : a.k_cache) +
                                      ((size_t)(blk * a.num_kv_heads + h) << a.log2_block) * D;
                float *sp = scale_of(a, blk, h, v);
                const float scale = grow_scale<D>(a, run, sp, run.fresh ? 0.f : *sp, __uint_as_float(top[j]), rows, lane);
                if (lane == 0) top[j] = __float_as_uint(scale);
            }
            __syncthreads();
            for (int row0 = 0; row0 < run.n; row0 += rows_at_once) {
                const int row = row0 + r;
                if (run.n > rows_at_once) plan(row);
                if (row >= run.n) continue;
                const size_t dst = (((size_t)(blk * a.num_kv_heads + h0) << a.log2_block) + off) * D;
                for (int h = head0; h < heads; h += head_step) {
                    const size_t at = dst + ((size_t)h << a.log2_block) * D;
                    float y[16];
                    key32(y, row, h);
                    store_codes(static_cast<unsigned char *>(a.k_cache) + at, xk, y, __uint_as_float(top[2 * h]));
                    const T *q = values + (row * heads + h) * D;
                    widen<T>(y, load_shared16(q + xv.a), load_shared16(q + xv.b));
                    store_codes(static_cast<unsigned char *>(a.v_cache) + at, xv, y, __uint_as_float(top[2 * h + 1]));
                }
            }
            __syncthreads();                                          // the slab and the scales are free again
        }
    }
}

// ---- host ---------------------------------------------------------------------------

// CTAs of a small 8-bit append at least: for runs, by fewer heads and then by
// fewer tokens to a CTA, until they do (one prompt of 1,000 tokens of 32/8
// heads: 7.0 us, 9.8 with four heads throughout; 64 sequences of four tokens:
// 7.4, 10.9 with whole blocks; more than these only delay what a decode step
// does in the CTAs after them), and for single tokens.
constexpr int kRunCtasByHeads = 256, kRunCtasByTokens = 152, kSingleCtas = 512;

template <int D, typename T>
cudaError_t launch_append(const RopeArgs &a, bool interleaved, bool fp8, cudaStream_t stream) {
    constexpr int UPR = D / 16;
    RopeArgs b = a;
    if (!fp8) {
        const unsigned long long units = (unsigned long long)a.num_tokens * (a.num_heads + 2 * a.num_kv_heads) * UPR;
        const unsigned grid = (unsigned)((units + kRopeThreads - 1) / kRopeThreads);
        return launch(interleaved ? rotary_append_kernel<D, T, true> : rotary_append_kernel<D, T, false>, dim3(grid),
                      dim3(kRopeThreads), 0, stream, b);
    }
    // single tokens
    b.single_tokens = a.num_tokens > 16 * kSingleCtas ? 16 : (a.num_tokens + kSingleCtas - 1) / kSingleCtas;
    constexpr int kRowsAtOnce = kAppend8Threads / UPR;
    b.single_parts = 1;
    while (b.single_parts * kRowsAtOnce < 2 * a.num_kv_heads && (long long)a.num_tokens * (b.single_parts + 1) <= kSingleCtas)
        b.single_parts++;
    b.single_ctas = ((a.num_tokens - 1) / b.single_tokens + 1) * b.single_parts;
    // longer runs
    const size_t head_bytes = (2 * sizeof(T) * D) << a.log2_block;   // of a block's keys and values
    b.group_heads = head_bytes < (size_t)kSlabBytes ? (int)(kSlabBytes / head_bytes) : 1;
    if (b.group_heads > a.num_kv_heads) b.group_heads = a.num_kv_heads;
    b.run_tokens = 1 << a.log2_block;
    const auto run_ctas = [&]() {
        return ((long long)a.num_tokens + b.run_tokens - 1) / b.run_tokens *
               ((a.num_kv_heads + b.group_heads - 1) / b.group_heads);
    };
    while (b.group_heads > 1 && run_ctas() < kRunCtasByHeads) b.group_heads = (b.group_heads + 1) / 2;
    while (b.run_tokens > 2 && run_ctas() < kRunCtasByTokens) b.run_tokens /= 2;
    b.run_ctas = (int)run_ctas();
    // queries, the runs mixed into the first half of them: what takes longest does not begin last
    const unsigned long long qunits =
        (unsigned long long)a.num_tokens * ((a.num_heads + kQueryRows - 1) / kQueryRows) * UPR;
    const unsigned long long q_ctas = (qunits + kAppend8Threads - 1) / kAppend8Threads;
    const unsigned long long among = b.run_ctas + q_ctas / 2;
    b.run_share = (((unsigned long long)b.run_ctas << 32) + among - 1) / among;
    auto kern = interleaved ? rotary_append8_kernel<D, T, true> : rotary_append8_kernel<D, T, false>;
    static std::atomic<unsigned long long> allowed[2];
    cudaError_t e = allow_smem(kern, 2 * kSlabBytes, allowed[interleaved]);
    if (e != cudaSuccess) return e;
    return launch(kern, dim3((unsigned)(b.single_ctas + b.run_ctas + q_ctas)), dim3(kAppend8Threads),
                  b.group_heads * head_bytes, stream, b);
}

pkv_status append_impl(const char *what, bool fp8, void *query_out, const void *query, const void *key,
                       const void *value, void *key_cache, void *value_cache, float *scales, const float *cos_sin,
                       const int32_t *positions, const int64_t *slot_mapping, int num_tokens, int num_heads,
                       int num_kv_heads, int head_dim, int rotary_dim, int num_positions, pkv_rotary_layout layout,
                       int64_t query_stride, int64_t key_stride, int64_t value_stride, int block_size, int num_blocks,
                       pkv_dtype dtype, cudaStream_t stream) {
    if (dtype != PKV_F16 && dtype != PKV_BF16) return fail(PKV_EINVAL, "%s: bad dtype %d", what, (int)dtype);
    if (layout != PKV_ROTARY_HALF && layout != PKV_ROTARY_INTERLEAVED)
        return fail(PKV_EINVAL, "%s: bad layout %d", what, (int)layout);
    if (head_dim != 64 && head_dim != 128)
        return fail(PKV_EINVAL, "%s: head_dim %d not supported (64 or 128)", what, head_dim);
    if (rotary_dim < 0 || rotary_dim % 16 || rotary_dim > head_dim || (!fp8 && rotary_dim == 0))
        return fail(PKV_EINVAL, "%s: rotary_dim %d not a multiple of 16 within the head of %d", what, rotary_dim,
                    head_dim);
    if (num_tokens < 0 || num_heads < 0 || num_kv_heads <= 0 || num_blocks < 0 || num_positions < 0 ||
        num_heads > 65536 || num_kv_heads > 65536)
        return fail(PKV_EINVAL, "%s: bad sizes (tokens %d, heads %d, kv heads %d, blocks %d, positions %d)", what,
                    num_tokens, num_heads, num_kv_heads, num_blocks, num_positions);
    if (!is_pow2(block_size) || block_size > (fp8 ? 128 : 1 << 20) || (fp8 && block_size < 4))
        return fail(PKV_EINVAL, "%s: block_size %d not a power of two%s", what, block_size, fp8 ? " in [4, 128]" : "");
    if (rotary_dim == 0 && num_heads > 0)
        return fail(PKV_EINVAL, "%s: queries given but nothing to rotate them by", what);
    if (num_tokens == 0) return PKV_OK;
    if (!key || !value || !key_cache || !value_cache || !slot_mapping || (fp8 && !scales) ||
        (num_heads > 0 && (!query || !query_out)) || (rotary_dim > 0 && (!cos_sin || !positions)))
        return fail(PKV_EINVAL, "%s: NULL pointer", what);
    if (!aligned16(key) || !aligned16(value) || !aligned16(key_cache) || !aligned16(value_cache) ||
        !aligned16(query) || !aligned16(query_out) || !aligned16(scales) || !aligned16(cos_sin))
        return fail(PKV_EINVAL, "%s: pointers must be 16-byte aligned", what);
    if ((num_heads > 0 && (query_stride < (int64_t)num_heads * head_dim || query_stride % 8)) ||
        key_stride < (int64_t)num_kv_heads * head_dim || key_stride % 8 ||
        value_stride < (int64_t)num_kv_heads * head_dim || value_stride % 8)
        return fail(PKV_EINVAL, "%s: token strides must be multiples of 8 elements that hold all heads "
                                "(query %lld, key %lld, value %lld)",
                    what, (long long)query_stride, (long long)key_stride, (long long)value_stride);
    if (num_heads > 0 && query_out == query && num_tokens > 1 && query_stride != (int64_t)num_heads * head_dim)
        return fail(PKV_EINVAL, "%s: queries %lld elements apart cannot be rotated in place", what, (long long)query_stride);
    // one CTA or thread per token and unit: the launch's grid is a 31-bit number
    const unsigned long long units =
        (unsigned long long)num_tokens * (num_heads + 2ull * num_kv_heads) * (unsigned)(head_dim / 16);
    if (units / 8 > 0x7fffffffull)
        return fail(PKV_EINVAL, "%s: %d tokens of %d + 2 x %d heads in one call", what, num_tokens, num_heads,
                    num_kv_heads);
    DeviceStatus *st = status_ptr();
    if (!st) return fail(PKV_ECUDA, "%s: no device status word", what);
    RopeArgs a;
    std::memset(&a, 0, sizeof a);
    a.q = query;
    a.k = key;
    a.v = value;
    a.q_out = query_out;
    a.k_cache = key_cache;
    a.v_cache = value_cache;
    a.scales = scales;
    a.cos_sin = cos_sin;
    a.positions = positions;
    a.slots = slot_mapping;
    a.st = st;
    a.q_stride = query_stride;
    a.k_stride = key_stride;
    a.v_stride = value_stride;
    a.num_slots = (int64_t)num_blocks * block_size;
    a.num_tokens = num_tokens;
    a.num_heads = num_heads;
    a.num_kv_heads = num_kv_heads;
    a.rot = rotary_dim;
    a.num_positions = num_positions;
    a.log2_block = ilog2(block_size);
    const bool il = layout == PKV_ROTARY_INTERLEAVED;
    cudaError_t e;
    if (head_dim == 128)
        e = dtype == PKV_BF16 ? launch_append<128, __nv_bfloat16>(a, il, fp8, stream)
                              : launch_append<128, __half>(a, il, fp8, stream);
    else
        e = dtype == PKV_BF16 ? launch_append<64, __nv_bfloat16>(a, il, fp8, stream)
                              : launch_append<64, __half>(a, il, fp8, stream);
    if (e != cudaSuccess) return fail(PKV_ECUDA, "%s: launch: %s", what, cudaGetErrorString(e));
    return PKV_OK;
}

}  // namespace
}  // namespace pkv

extern "C" {

pkv_status rotary_table(float *cos_sin, int num_positions, int rotary_dim, double base, pkv_rotary_scaling scaling,
                        double factor, int original_positions, double low_turns, double high_turns, double magnitude,
                        struct CUstream_st *stream) {
    using namespace pkv;
    if (num_positions < 0 || num_positions > kMaxPositions || rotary_dim <= 0 || rotary_dim % 16 ||
        rotary_dim > kMaxRotaryDim)
        return fail(PKV_EINVAL, "rotary_table: bad sizes (%d positions: up to %d, rotary_dim %d: a multiple of 16 up to %d)",
                    num_positions, kMaxPositions, rotary_dim, kMaxRotaryDim);
    if (!(base > 1.0) || !std::isfinite(base) || !(std::fabs(magnitude) <= (double)FLT_MAX))
        return fail(PKV_EINVAL, "rotary_table: base %g must be above 1, magnitude %g finite in fp32", base, magnitude);
    if (scaling != PKV_ROTARY_UNSCALED && scaling != PKV_ROTARY_LINEAR && scaling != PKV_ROTARY_BY_PARTS)
        return fail(PKV_EINVAL, "rotary_table: bad scaling %d", (int)scaling);
    if (scaling != PKV_ROTARY_UNSCALED && (!(factor >= 1.0) || !std::isfinite(factor)))
        return fail(PKV_EINVAL, "rotary_table: scaling factor %g below 1", factor);
    if (scaling == PKV_ROTARY_BY_PARTS &&
        (original_positions <= 0 || !(high_turns > low_turns) || !std::isfinite(high_turns) || !std::isfinite(low_turns)))
        return fail(PKV_EINVAL, "rotary_table: scaling by parts needs the original positions (%d) and low turns (%g) "
                                "below high turns (%g)",
                    original_positions, low_turns, high_turns);
    if (num_positions == 0) return PKV_OK;
    if (!cos_sin || !aligned16(cos_sin))
        return fail(PKV_EINVAL, "rotary_table: the table must be a 16-byte aligned device pointer");
    TurnTable tab;
    std::memset(&tab, 0, sizeof tab);
    constexpr double kTwoPi = 6.283185307179586476925286766559;
    for (int i = 0; i < rotary_dim / 2; i++) {
        double theta = std::pow(base, -2.0 * i / rotary_dim);
        if (scaling == PKV_ROTARY_LINEAR) {
            theta /= factor;
        } else if (scaling == PKV_ROTARY_BY_PARTS) {
            // pairs that turn often over the original positions keep their angle, slow ones are stretched
            const double turns = original_positions * theta / kTwoPi;
            double keep = (turns - low_turns) / (high_turns - low_turns);
            keep = keep < 0.0 ? 0.0 : keep > 1.0 ? 1.0 : keep;
            theta = theta * (keep + (1.0 - keep) / factor);
        }
        tab.turn[i] = (unsigned long long)std::nearbyint(theta / kTwoPi * 0x1p64);   // theta <= 1: below 2^62
    }
    const int columns = rotary_dim / 4, rows = kRopeThreads / columns;
    // one wave of CTAs for long tables, since fetching the turns costs each CTA about a microsecond (131,072 x 128:
    // 7 us more with 32 positions to a CTA); at least four positions to a thread in short ones
    const int wave = (sm_count() > 0 ? sm_count() : 1) * 8;
    int per_cta = (num_positions + wave - 1) / wave;
    per_cta = per_cta < 4 * rows ? 4 * rows : (per_cta + rows - 1) / rows * rows;
    const long long ctas = ((long long)num_positions + per_cta - 1) / per_cta;
    cudaError_t e = launch(rotary_table_kernel, dim3((unsigned)ctas), dim3(kRopeThreads), 0, stream,
                           reinterpret_cast<float4 *>(cos_sin), tab, num_positions, columns, rows, per_cta,
                           (float)magnitude);
    if (e != cudaSuccess) return fail(PKV_ECUDA, "rotary_table: launch: %s", cudaGetErrorString(e));
    return PKV_OK;
}

pkv_status kv_rotary_and_cache(void *query_out, const void *query, const void *key, const void *value,
                               void *key_cache, void *value_cache, const float *cos_sin, const int32_t *positions,
                               const int64_t *slot_mapping, int num_tokens, int num_heads, int num_kv_heads,
                               int head_dim, int rotary_dim, int num_positions, pkv_rotary_layout layout,
                               int64_t query_stride, int64_t key_stride, int64_t value_stride, int block_size,
                               int num_blocks, pkv_dtype dtype, struct CUstream_st *stream) {
    return pkv::append_impl("kv_rotary_and_cache", false, query_out, query, key, value, key_cache, value_cache, nullptr,
                            cos_sin, positions, slot_mapping, num_tokens, num_heads, num_kv_heads, head_dim, rotary_dim,
                            num_positions, layout, query_stride, key_stride, value_stride, block_size, num_blocks, dtype,
                            stream);
}

pkv_status kv_rotary_and_cache_fp8(void *query_out, const void *query, const void *key, const void *value,
                                   void *key_cache, void *value_cache, float *scales, const float *cos_sin,
                                   const int32_t *positions, const int64_t *slot_mapping, int num_tokens,
                                   int num_heads, int num_kv_heads, int head_dim, int rotary_dim, int num_positions,
                                   pkv_rotary_layout layout, int64_t query_stride, int64_t key_stride,
                                   int64_t value_stride, int block_size, int num_blocks, pkv_dtype dtype,
                                   struct CUstream_st *stream) {
    return pkv::append_impl("kv_rotary_and_cache_fp8", true, query_out, query, key, value, key_cache, value_cache,
                            scales, cos_sin, positions, slot_mapping, num_tokens, num_heads, num_kv_heads, head_dim,
                            rotary_dim, num_positions, layout, query_stride, key_stride, value_stride, block_size,
                            num_blocks, dtype, stream);
}

}  // extern "C"
