// A key-value cache held in 4 bits: writing bf16 rows in, reading them back,
// and the decode attention that reads it (sm_103a).
//
// A row of 128 channels is two halves of 64.  Half h has a bf16 minimum m and
// a bf16 scale s = bf16((max - m) / 15); a code u = clamp(rint((x - m) / s),
// 0, 15) stands for m + s u.  Byte 8r + j of the row's 64 holds channels
// 8r + 2j (low nibble) and 8r + 2j + 1 for j < 4, and the same channels + 64
// in byte 8r + 4 + j: eight units of 8 bytes, each with one 32-bit word per
// half.  Parameters: bf16 [n_kv][max_pos][2][2], (s, m) per half.
#include <algorithm>
#include <cmath>
#include <cstdio>
#include <mutex>

#include "fourbit.cuh"
#include "tts_decode.h"

namespace tts {
namespace {

constexpr int kRowBytes = 64;
constexpr int kMaxSplitUnits = 160;  // split partials per kv head x kv heads, about one per SM
constexpr int kKv4MaxPos = 1 << 20;
constexpr int kKv4MaxHeads = 4096;   // query heads
constexpr int kKv4MaxKvHeads = 1024;
constexpr size_t kTicketBytes = 4 * kKv4MaxKvHeads;  // the workspace's first bytes, whatever the heads

// cos and sin of the position's angles in fp64, as an fp32 value and the rest.
struct RopeRow {
    float2 cs[kHeadDim / 2], rest[kHeadDim / 2];
};

struct Kv4Params {
    const float* qkv;
    const __nv_bfloat16 *q_norm, *k_norm;
    uint8_t *k4, *v4;
    uint32_t *k_par, *v_par;  // [n_kv][max_pos][2] words: (s, m) of one half, s in the low 16 bits
    float* out;
    float* kv_row;
    int n_q, n_kv, max_pos, pos;
    float eps;
    int S, tiles_per_split;  // splits per kv head, tiles of 16 cached positions per split
    int cluster;             // a head's splits are a cluster, joined through shared memory
    int halves;              // 1: a kv head's queries are two heads
    unsigned* tickets;       // [n_kv], zero between calls
    float2* part_ml;         // [n_kv][S][G] maximum, sum
    float* part_o;           // [n_kv][S][G][128]
    RopeRow rope;
};

// fp32 bits in the order of the values, as a signed integer, and back.
__device__ __forceinline__ int ordered(float x) {
    const int b = __float_as_int(x);
    return b ^ ((b >> 31) & 0x7fffffff);
}
__device__ __forceinline__ float from_ordered(int b) { return __int_as_float(b ^ ((b >> 31) & 0x7fffffff)); }

// Quantise one row held by a warp: lane l has channels 4l .. 4l + 3 (bf16
// values), so lanes 0-15 hold half 0 and lanes 16-31 half 1.  Returns the
// lane's four codes in 16 bits; *par is its half's parameter word.  The
// arithmetic is IEEE fp32 as defined above.  A half whose range is not finite
// (it holds a NaN or an infinity) gets NaN parameters: its values read as NaN.
__device__ __forceinline__ uint32_t quant_row(const float x[4], uint32_t* par) {
    const unsigned half = (threadIdx.x & 16) ? 0xffff0000u : 0x0000ffffu;
    const int lo4 = min(min(ordered(x[0]), ordered(x[1])), min(ordered(x[2]), ordered(x[3])));
    const int hi4 = max(max(ordered(x[0]), ordered(x[1])), max(ordered(x[2]), ordered(x[3])));
    // + 0: a minimum of -0 is stored as 0.  NaN and infinities sort to the ends
    const float lo = from_ordered(__reduce_min_sync(half, lo4)) + 0.f, hi = from_ordered(__reduce_max_sync(half, hi4));
    const __nv_bfloat16 sb = __float2bfloat16_rn(__fdiv_rn(hi - lo, 15.f));
    const float s = __bfloat162float(sb);
    if (!isfinite(s)) {
        *par = 0x7fff7fffu;
        return 0;
    }
    // quotients by one reciprocal; below 2^-60 numerator and divisor are scaled
    // so that the reciprocal stays finite
    const float k = s < 0x1p-60f ? 0x1p100f : 1.f, ks = s * k, rs = __frcp_rn(ks);
    uint32_t code = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float q = s > 0.f ? fminf(fmaxf(rintf(div_rn_by((x[j] - lo) * k, ks, rs)), 0.f), 15.f) : 0.f;
        code |= (uint32_t)q << (4 * j);
    }
    *par = (uint32_t)__bfloat16_as_ushort(sb) | (__float_as_uint(lo) & 0xffff0000u);
    return code;
}
// Byte offset in a row of lane l's two bytes.
__device__ __forceinline__ int lane_byte(int lane) {
    return 8 * ((lane & 15) >> 1) + 4 * (lane >> 4) + 2 * (lane & 1);
}
__device__ __forceinline__ void store_row(uint32_t code, uint32_t par, uint8_t* row, uint32_t* par_row, int lane) {
    *reinterpret_cast<uint16_t*>(row + lane_byte(lane)) = (uint16_t)code;
    if ((lane & 15) == 0) par_row[lane >> 4] = par;
}
// ---- rows in and out ------------------------------------------------------------
// Bound by memory (256 bytes of bf16 and 72 of codes and parameters a row).
// A row is 16 lanes', 8 channels each: 16-byte accesses on the bf16 side, one
// word of codes (a unit's share of a half) on the other.  A thread keeps
// kRowsAhead rows in flight.
constexpr int kRowThreads = 256;
constexpr int kRowsAhead = 4;
constexpr int kBlockRows = kRowThreads / 16 * kRowsAhead;

struct RowParams {
    const uint8_t *k4, *v4;
    const uint32_t *k_par, *v_par;
    const uint16_t *k, *v;
    int p0, np, stride, max_pos;  // positions [p0, p0 + np); rows a head of the bf16 caches, of the 4-bit one
};

__device__ __forceinline__ __nv_bfloat162 as_bf162(uint32_t w) { return *reinterpret_cast<const __nv_bfloat162*>(&w); }
__device__ __forceinline__ uint32_t as_u32(__nv_bfloat162 v) { return *reinterpret_cast<const uint32_t*>(&v); }

__global__ void __launch_bounds__(kRowThreads) quantize_kv4_kernel(const RowParams p) {
    pdl_trigger();
    pdl_wait();
    const int head = blockIdx.y >> 1, lane = threadIdx.x & 15, h = lane >> 3, unit = lane & 7;
    const bool is_v = blockIdx.y & 1;
    const int i0 = blockIdx.x * kBlockRows + (threadIdx.x >> 4);
    const uint16_t* src = (is_v ? p.v : p.k) + ((size_t)head * p.stride + p.p0) * kHeadDim + 8 * lane;
    uint4 x[kRowsAhead];
#pragma unroll
    for (int j = 0; j < kRowsAhead; ++j) {
        const int i = min(i0 + 16 * j, p.np - 1);  // past the end the last row again, not stored
        x[j] = *reinterpret_cast<const uint4*>(src + (size_t)i * kHeadDim);
    }
#pragma unroll
    for (int j = 0; j < kRowsAhead; ++j) {
        const int i = i0 + 16 * j;
        const uint32_t w[4] = {x[j].x, x[j].y, x[j].z, x[j].w};
        // minimum and maximum of the half, as one minimum of (x, -x); NaN stays NaN
        __nv_bfloat162 mn = __hmin2_nan(__hmin2_nan(as_bf162(w[0]), as_bf162(w[1])), __hmin2_nan(as_bf162(w[2]), as_bf162(w[3])));
        __nv_bfloat162 mx = __hmax2_nan(__hmax2_nan(as_bf162(w[0]), as_bf162(w[1])), __hmax2_nan(as_bf162(w[2]), as_bf162(w[3])));
        __nv_bfloat162 both = __halves2bfloat162(__hmin_nan(__low2bfloat16(mn), __high2bfloat16(mn)),
                                                 __hneg(__hmax_nan(__low2bfloat16(mx), __high2bfloat16(mx))));
#pragma unroll
        for (int d = 1; d <= 4; d <<= 1) both = __hmin2_nan(both, as_bf162(__shfl_xor_sync(0xffffffffu, as_u32(both), d)));
        const float lo = __low2float(both) + 0.f, hi = -__high2float(both);  // + 0: a minimum of -0 is stored as 0
        // s, its reciprocal and the quotients by one FMA correction each, IEEE results
        // as quant_row's; very small ranges, where that does not hold, the slow way
        const float range = hi - lo;
        uint32_t code = 0, par = 0x7fff7fffu;
        if (range >= 0x1p-50f && isfinite(range)) {
            constexpr float kFifteenth = 1.f / 15.f;
            const __nv_bfloat16 sb = __float2bfloat16_rn(div_rn_by(range, 15.f, kFifteenth));
            const float s = __bfloat162float(sb), rs = __frcp_rn(s);
            if (isfinite(s)) par = (uint32_t)__bfloat16_as_ushort(sb) | (__float_as_uint(lo) & 0xffff0000u);
            const f32x2 ml = pack2(-lo, -lo), ms = pack2(-s, -s), rr = pack2(rs, rs);
            // 1.5 2^23 added and taken away rounds to the nearest even integer; s has 8
            // bits of (max - min) / 15, so no quotient rounds above 15
            const f32x2 magic = pack2(12582912.f, 12582912.f), back = pack2(-12582912.f, -12582912.f);
            float u[8];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const f32x2 d = add2(pack2(bf16lo(w[c]), bf16hi(w[c])), ml), q0 = mul2(d, rr);
                const f32x2 q = fma2(fma2(q0, ms, d), rr, q0);
                const float2 n = unpack2(add2(add2(q, magic), back));
                u[2 * c] = n.x;
                u[2 * c + 1] = n.y;
            }
            // four codes as one exact integer below 2^16, in the low bits of 2^23 + it
            const float c0 = fmaf(4096.f, u[3], fmaf(256.f, u[2], fmaf(16.f, u[1], u[0]))) + 8388608.f;
            const float c1 = fmaf(4096.f, u[7], fmaf(256.f, u[6], fmaf(16.f, u[5], u[4]))) + 8388608.f;
            code = isfinite(s) ? __byte_perm(__float_as_uint(c0), __float_as_uint(c1), 0x5410) : 0u;
        } else if (isfinite(range)) {
            const __nv_bfloat16 sb = __float2bfloat16_rn(__fdiv_rn(range, 15.f));
            const float s = __bfloat162float(sb);
            par = (uint32_t)__bfloat16_as_ushort(sb) | (__float_as_uint(lo) & 0xffff0000u);
            const float ks = s * 0x1p100f, rs = __frcp_rn(ks);
            for (int c = 0; c < 8 && s > 0.f; ++c) {
                const float v = __uint_as_float(c & 1 ? w[c >> 1] & 0xffff0000u : w[c >> 1] << 16);
                code |= (uint32_t)fminf(rintf(div_rn_by((v - lo) * 0x1p100f, ks, rs)), 15.f) << (4 * c);
            }
        }
        if (i < p.np) {
            const size_t at = (size_t)head * p.max_pos + p.p0 + i;
            uint8_t* row = const_cast<uint8_t*>(is_v ? p.v4 : p.k4) + at * kRowBytes;
            *reinterpret_cast<uint32_t*>(row + 8 * unit + 4 * h) = code;
            if (unit == 0) const_cast<uint32_t*>(is_v ? p.v_par : p.k_par)[at * 2 + h] = par;
        }
    }
}

__global__ void __launch_bounds__(kRowThreads) dequantize_kv4_kernel(const RowParams p) {
    pdl_trigger();
    pdl_wait();
    const int head = blockIdx.y >> 1, lane = threadIdx.x & 15, h = lane >> 3, unit = lane & 7;
    const bool is_v = blockIdx.y & 1;
    const int i0 = blockIdx.x * kBlockRows + (threadIdx.x >> 4);
    const size_t first = (size_t)head * p.max_pos + p.p0;
    const uint8_t* codes = (is_v ? p.v4 : p.k4) + first * kRowBytes + 8 * unit + 4 * h;
    const uint32_t* pars = (is_v ? p.v_par : p.k_par) + first * 2 + h;
    uint16_t* dst = const_cast<uint16_t*>(is_v ? p.v : p.k) + ((size_t)head * p.stride + p.p0) * kHeadDim + 8 * lane;
    uint32_t code[kRowsAhead], par[kRowsAhead];
#pragma unroll
    for (int j = 0; j < kRowsAhead; ++j) {
        const int i = min(i0 + 16 * j, p.np - 1);
        code[j] = *reinterpret_cast<const uint32_t*>(codes + (size_t)i * kRowBytes);
        par[j] = pars[(size_t)i * 2];
    }
#pragma unroll
    for (int j = 0; j < kRowsAhead; ++j) {
        const int i = i0 + 16 * j;
        // a nibble in a 16-bit half is the fp16 subnormal u 2^-24: scale and minimum in
        // one FMA (s 2^24 is exact but for the largest scales, which go the long way)
        const float s = bf16lo(par[j]), m = bf16hi(par[j]);
        const bool large = !(fabsf(s) < 0x1p100f);
        const f32x2 ss = large ? pack2(s, s) : pack2(s * 16777216.f, s * 16777216.f), mm = pack2(m, m);
        float2 f[4];  // channels (0, 4), (1, 5), (2, 6), (3, 7)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const uint32_t u = (code[j] >> (4 * c)) & 0x000f000fu;
            float2 x = __half22float2(*reinterpret_cast<const __half2*>(&u));
            if (large) x = make_float2(x.x * 16777216.f, x.y * 16777216.f);
            f[c] = unpack2(fma2(pack2(x.x, x.y), ss, mm));
        }
        const uint32_t w[4] = {as_u32(__floats2bfloat162_rn(f[0].x, f[1].x)), as_u32(__floats2bfloat162_rn(f[2].x, f[3].x)),
                               as_u32(__floats2bfloat162_rn(f[0].y, f[1].y)), as_u32(__floats2bfloat162_rn(f[2].y, f[3].y))};
        if (i < p.np) *reinterpret_cast<uint4*>(dst + (size_t)i * kHeadDim) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// q/k RMSNorm over the head then rotate-half RoPE: lane l has channels
// 4l .. 4l + 3, whose rotation partners sit in lane l ^ 16.
__device__ __forceinline__ void norm_rope(float4 x, uint2 gb, const float4* rope, float eps, int lane, float o[4]) {
    const float ss = warp_sum(x.x * x.x + x.y * x.y + x.z * x.z + x.w * x.w);
    const float r = 1.0f / sqrtf(ss / (float)kHeadDim + eps);
    const float a[4] = {x.x * r * bf16lo(gb.x), x.y * r * bf16hi(gb.x), x.z * r * bf16lo(gb.y), x.w * r * bf16hi(gb.y)};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float partner = __shfl_xor_sync(0xffffffffu, a[j], 16);
        const float4 cs = rope[(4 * lane + j) & 63];
        o[j] = lane < 16 ? a[j] * cs.x - partner * cs.y : a[j] * cs.x + partner * cs.y;
    }
}

// The same to about 2^-44, for the new key: its 4-bit codes are a step
// function of it and must not depend on the order of an fp32 sum.  Numbers are
// unevaluated sums hi + lo of two fp32 (Dekker's and Knuth's error-free
// product and sum); the fp64 unit took 6 us for these 128 channels.
struct Two {
    float hi, lo;
};
__device__ __forceinline__ Two two_sum(float a, float b) {
    const float s = __fadd_rn(a, b), t = __fsub_rn(s, a);
    return {s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t))};
}
__device__ __forceinline__ Two two_prod(float a, float b) {
    const float p = __fmul_rn(a, b);
    return {p, __fmaf_rn(a, b, -p)};
}
__device__ __forceinline__ Two renorm(float hi, float lo) {
    const float s = __fadd_rn(hi, lo);
    return {s, __fsub_rn(lo, __fsub_rn(s, hi))};
}
__device__ __forceinline__ Two add(Two a, Two b) {
    const Two s = two_sum(a.hi, b.hi);
    return renorm(s.hi, __fadd_rn(s.lo, __fadd_rn(a.lo, b.lo)));
}
__device__ __forceinline__ Two mul(Two a, Two b) {
    const Two p = two_prod(a.hi, b.hi);
    return renorm(p.hi, __fadd_rn(p.lo, __fmaf_rn(a.hi, b.lo, __fmul_rn(a.lo, b.hi))));
}
__device__ __forceinline__ void norm_rope_exact(float4 x4, uint2 gb, const float4* rope, float eps, int lane,
                                                float o[4]) {
    const float x[4] = {x4.x, x4.y, x4.z, x4.w};
    const float gn[4] = {bf16lo(gb.x), bf16hi(gb.x), bf16lo(gb.y), bf16hi(gb.y)};
    Two ss = add(add(two_prod(x[0], x[0]), two_prod(x[1], x[1])), add(two_prod(x[2], x[2]), two_prod(x[3], x[3])));
#pragma unroll
    for (int d = 16; d > 0; d >>= 1)
        ss = add(ss, Two{__shfl_xor_sync(0xffffffffu, ss.hi, d), __shfl_xor_sync(0xffffffffu, ss.lo, d)});
    const Two v = add(Two{ss.hi * (1.f / kHeadDim), ss.lo * (1.f / kHeadDim)}, Two{eps, 0.f});
    // 1 / sqrt(v): an fp32 value y corrected by Newton's step on e = 1 - v y^2
    const float y = 1.0f / sqrtf(v.hi);
    const Two vy2 = mul(v, two_prod(y, y));
    const float e = __fsub_rn(__fsub_rn(1.f, vy2.hi), vy2.lo);
    const Two rs{y, y * e * (0.5f + 0.375f * e)};
    Two a[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) a[j] = mul(two_prod(x[j], gn[j]), rs);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const Two partner{__shfl_xor_sync(0xffffffffu, a[j].hi, 16), __shfl_xor_sync(0xffffffffu, a[j].lo, 16)};
        const float4 cs = rope[(4 * lane + j) & 63];
        const float sg = lane < 16 ? -1.f : 1.f;
        o[j] = add(mul(a[j], Two{cs.x, cs.z}), mul(partner, Two{sg * cs.y, sg * cs.w})).hi;
    }
}

// ---- the attention kernel -------------------------------------------------------
// A block takes one kv head and one contiguous range of 16-position tiles (a
// split); its warps take the range's tiles in turn, each with its own ring of
// asynchronous copies, running maximum, sum and output, so nothing in the loop
// waits for another warp.  The partials are joined in a fixed order: a block's
// warps in its shared memory, and the blocks of a head, where they are a cluster, by
// writing each a share of the channels into one another's shared memory, else
// through the workspace by the last block to finish.
//
// Both products run on the tensor cores (m16n8k16, fp16 operands, fp32 sums).
// Codes enter centred, u - 8 and, from a whole byte, (u - 8) + 16 (u' - 8), exact
// in fp16 (nibble_bytes and the next): one logical and one fp16 instruction per
// two of them.  The even code is taken out of the byte on the other operand
// (scores) or in the epilogue (output), and a half's minimum counts as
// m + 8 s: with m and u the sums of values that cancel over the positions grew to
// 200 times the result at 65536 positions, and its error to 1e-4 (2e-6 with V
// codes all centred at 8, half a step off the middle).
//   scores  A = K codes (16 positions), B = queries.  score = sum over halves of
//           s_K q . (u - 8) + (m_K + 8 s_K) sum(q): a position's scale and
//           centre enter in fp32 on the accumulators.
//   output  A = V codes (16 channels of a half), B = p s_V of 16 positions;
//           sum of p (m_V + centre s_V) beside it in fp32.
// The other operand is fp32 in two fp16 parts, of a value scaled by a power of
// two towards fp16's upper end: 22 bits, and for small ones a floor of 2^-39
// (queries) or 2^-33 (weights) of the largest, so nothing falls below fp32
// accuracy by more than the rounding of the sums.  Up to four query
// heads sit side by side with their low parts in the product's eight columns;
// eight heads take a product for each part.  The scaling of the weights
// follows their running maximum per head and half, like the softmax maximum.
// (Queries and weights as A, codes as B was measured first: the same integer
// work, but 32 products a tile instead of 16 and 96 registers of operands and
// sums instead of 48, so 12 warps an SM instead of 16.)
constexpr int kAttnWarps = 16;
constexpr int kTilePos = 16;
constexpr int kStages = 3;
constexpr int kStageV = kTilePos * kRowBytes;             // K rows, then V rows (permuted)
constexpr int kStagePar = 2 * kStageV;                    // then K and V parameters
constexpr int kStageBytes = kStagePar + 2 * kTilePos * 8;
constexpr int kRingBytes = kStages * kStageBytes;         // per warp
constexpr int kAttnSmem = kAttnWarps * kRingBytes;
constexpr int kMaxCluster = 16;    // blocks of a cluster, at most
constexpr int kOneBlockTiles = 12;  // a head of up to so many tiles is one block's
constexpr int kClusterTiles = 4;    // tiles a block of a cluster, at least
static_assert(kRingBytes >= 8 * kHeadDim * 4, "a warp's output partial reuses its ring");

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async16_zfill(uint32_t dst, const void* src, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async8_zfill(uint32_t dst, const void* src, int bytes) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ void mma16816(float c[4], const uint32_t a[4], uint2 b) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b.x), "r"(b.y));
}
// c = A B, without clearing c first
__device__ __forceinline__ void mma16816_first(float c[4], const uint32_t a[4], uint2 b) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b.x), "r"(b.y), "f"(0.f));
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// Two values as fp16 (x in the low half), and what fp16 left of them.
__device__ __forceinline__ void split_h2(float x, float y, uint32_t* hi, uint32_t* lo) {
    const __half2 h = __floats2half2_rn(x, y);
    const float2 f = __half22float2(h);
    const __half2 r = __floats2half2_rn(x - f.x, y - f.y);
    *hi = *reinterpret_cast<const uint32_t*>(&h);
    *lo = *reinterpret_cast<const uint32_t*>(&r);
}
// The transpose of an 8 x 8 matrix of 16-bit values held by a warp, lane
// (row, pair of columns).
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}
// The biased exponent of w >= 0, at least 15, and the power of two that takes
// w to [2^14, 2^15).
__device__ __forceinline__ int expo(float w) { return max((int)(__float_as_uint(w) >> 23), 15); }
__device__ __forceinline__ float pow2_field(int field) { return __uint_as_float((uint32_t)field << 23); }
__device__ __forceinline__ float to_2p15(int e) { return pow2_field(268 - e); }
// For the weights, to [2^8, 2^9): six more doublings fit before fp16 ends, so
// that a weight above all before it seldom moves the scale (measured: with
// none to spare every second tile of normal data did), and the floor of the
// low parts is still 2^-33 of the largest weight.
__device__ __forceinline__ float to_2p9(int e) { return pow2_field(262 - e); }
__device__ __forceinline__ int expo_of(float to) { return 262 - (int)(__float_as_uint(to) >> 23); }

// A lane's share of a tile's copies: codes of both caches (two 16-byte pieces
// each) and one row's 8 parameter bytes (a head's parameters start on 8 bytes
// only when max_pos is odd; lanes 0-15 K, 16-31 V).  Rows at and past n read
// as zero and are not touched in memory.
struct LaneCopy {
    const uint8_t *k, *v, *par;  // at tile 0
    uint32_t k_dst, v_dst[2], par_dst;
    int n;
    __device__ __forceinline__ LaneCopy(const Kv4Params& p, size_t base, uint32_t ring, int lane) {
        k = p.k4 + base * kRowBytes + lane * 16;
        v = p.v4 + base * kRowBytes + lane * 16;
        par = reinterpret_cast<const uint8_t*>((lane < 16 ? p.k_par : p.v_par) + (base + (lane & 15)) * 2);
        n = p.pos;
        k_dst = ring + lane * 16;
        // V: rows 2 t + (0, 1, 8, 9) at column pair t of four lines, so that the
        // 8-byte reads of the output product touch every bank once
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int idx = lane + 32 * i, row = idx >> 2, c = idx & 3;
            const int line = ((row & 1) + 2 * (row >> 3)) * 2 + (c >> 1), slot = 2 * ((row >> 1) & 3) + (c & 1);
            v_dst[i] = ring + kStageV + line * 128 + slot * 16;
        }
        par_dst = ring + kStagePar + lane * 8;
    }
    __device__ __forceinline__ void issue(int tile, int stage, int lane) const {
        const size_t off = (size_t)tile * (kTilePos * kRowBytes);
        const uint32_t s = stage * kStageBytes;
        const int left = n - tile * kTilePos;
        if (left >= kTilePos) {
            cp_async16(k_dst + s, k + off);
            cp_async16(k_dst + s + 512, k + off + 512);
            cp_async16(v_dst[0] + s, v + off);
            cp_async16(v_dst[1] + s, v + off + 512);
            cp_async8_zfill(par_dst + s, par + (size_t)tile * (kTilePos * 8), 8);
        } else {
            const int b0 = (lane >> 2) < left ? 16 : 0, b1 = (lane >> 2) + 8 < left ? 16 : 0;
            const int bp = (lane & 15) < left ? 8 : 0;
            // a copy of no bytes still wants an address inside the cache: row 0's
            const uint8_t *k0 = b0 ? k + off : k - lane * 16, *k1 = b1 ? k + off + 512 : k - lane * 16;
            const uint8_t *v0 = b0 ? v + off : v - lane * 16, *v1 = b1 ? v + off + 512 : v - lane * 16;
            cp_async16_zfill(k_dst + s, k0, b0);
            cp_async16_zfill(k_dst + s + 512, k1, b1);
            cp_async16_zfill(v_dst[0] + s, v0, b0);
            cp_async16_zfill(v_dst[1] + s, v1, b1);
            cp_async8_zfill(par_dst + s, bp ? par + (size_t)tile * (kTilePos * 8) : par - (lane & 15) * 8, bp);
        }
    }
};

// To the same place in the shared memory of block `rank` of the cluster.
__device__ __forceinline__ uint32_t remote(const void* at, int rank) {
    uint32_t a;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(at)), "r"(rank));
    return a;
}
__device__ __forceinline__ void store_remote(float2* at, int rank, float2 v) {
    asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(remote(at, rank)), "f"(v.x), "f"(v.y) : "memory");
}
__device__ __forceinline__ void store_remote(float4* at, int rank, float4 v) {
    asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(remote(at, rank)), "f"(v.x), "f"(v.y), "f"(v.z),
                 "f"(v.w)
                 : "memory");
}

template <int G>
__global__ void __launch_bounds__(kAttnWarps * 32, 1) attn_kv4_kernel(const __grid_constant__ Kv4Params p) {
    extern __shared__ __align__(128) uint8_t ring[];
    __shared__ float4 rope[kHeadDim / 2];             // (cos, sin, rest of cos, rest of sin)
    __shared__ __align__(16) float qs[G][kHeadDim];   // log2(e) / sqrt(128) times the rotated queries
    constexpr bool kPack = G <= 4;      // high and low parts in one product's columns
    constexpr int kParts = kPack ? 1 : 2;
    __shared__ uint2 frag[kParts][4][2][32];          // the scores' query operand, by lane
    __shared__ float qhead[G][3];                     // sums over the halves, 1 over the operand's power of two
    __shared__ __align__(16) float vnew[kHeadDim];    // the new value row as cached
    __shared__ float wm[kAttnWarps + 1][G], wl[kAttnWarps + 1][G];
    __shared__ float merge_c[kMaxSplitUnits][G];      // a partial's weight in the merge
    __shared__ float merge_l[G];
    __shared__ int s_last;
    // a cluster's partials of this block's share of the outputs
    __shared__ __align__(16) float4 box_o[G * kHeadDim / 4 + kMaxCluster];
    __shared__ float2 box_ml[kMaxCluster][G];

    // the warp's number by a shuffle: the compiler then keeps the loop's control in
    // uniform registers
    const int lane = threadIdx.x & 31, warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);
    const int r = lane >> 2, t = lane & 3;
    const int g = blockIdx.x, split = blockIdx.y;
    if (p.cluster) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
    const bool has_new = split == p.S - 1;
    const int kv = g >> p.halves;  // its head of the cache
    const size_t base = (size_t)kv * p.max_pos;
    const int tile_end = min((p.pos + kTilePos - 1) / kTilePos, (split + 1) * p.tiles_per_split);

    // the angles from the launch parameters to shared memory, an entry a warp at
    // a time: parameters are read fast at one address a warp only
    constexpr int kEach = (kHeadDim / 2 + kAttnWarps - 1) / kAttnWarps;
    float2 cs[kEach], rest[kEach];
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        const int at = min(warp + i * kAttnWarps, kHeadDim / 2 - 1);
        cs[i] = p.rope.cs[at];
        rest[i] = p.rope.rest[at];
    }
    if (lane == 0) {
#pragma unroll
        for (int i = 0; i < kEach; ++i)
            rope[min(warp + i * kAttnWarps, kHeadDim / 2 - 1)] = make_float4(cs[i].x, cs[i].y, rest[i].x, rest[i].y);
    }
    pdl_trigger();
    pdl_wait();
    // the group's queries, one warp each, and in the last split the new row, its
    // key by the last warp and its value by the one before: their loads first
    const bool new_k = has_new && warp == kAttnWarps - 1, new_v = has_new && warp == kAttnWarps - 2;
    float4 x = {};
    uint2 gain = {};
    if (warp < G || new_k || new_v) {
        const int vec = new_v ? p.n_q + p.n_kv + kv : new_k ? p.n_q + kv : g * G + warp;
        x = reinterpret_cast<const float4*>(p.qkv)[(size_t)vec * (kHeadDim / 4) + lane];
        gain = reinterpret_cast<const uint2*>(new_k ? p.k_norm : p.q_norm)[lane];
    }
    uint8_t* my_ring = ring + warp * kRingBytes;
    const LaneCopy copy(p, base, smem_u32(my_ring), lane);
    int next = split * p.tiles_per_split + warp;  // next tile to copy
    if (next < tile_end) copy.issue(next, 0, lane);
    cp_async_commit();
    next += kAttnWarps;
    __syncthreads();
    // the other stages' copies only now: before it they held up the loads above
#pragma unroll
    for (int s = 1; s < kStages - 1; ++s) {
        if (next < tile_end) copy.issue(next, s, lane);
        cp_async_commit();
        next += kAttnWarps;
    }
    if (warp < G) {
        float q[4];
        norm_rope(x, gain, rope, p.eps, lane, q);
        const float c = 1.4426950408889634f / sqrtf((float)kHeadDim);
#pragma unroll
        for (int j = 0; j < 4; ++j) q[j] *= c;
        reinterpret_cast<float4*>(qs[warp])[lane] = make_float4(q[0], q[1], q[2], q[3]);
        // the scores' operand.  Word w of a K row's 16-byte piece t holds channels
        // 64 (w % 2) + 8 (2 t + w / 2) + 0..7; nibbles (0, 4) and (1, 5) are one
        // product's rows, (2, 6) and (3, 7) the other's.  Codes come as an even
        // nibble u and the whole byte u + 16 u': q u + q' u' = (q - q'/16) u +
        // (q'/16) (u + 16 u')
        const unsigned amax = __reduce_max_sync(
            0xffffffffu, __float_as_uint(fmaxf(fmaxf(fabsf(q[0]), fabsf(q[1])), fmaxf(fabsf(q[2]), fabsf(q[3])))));
        const int e = expo(__uint_as_float(amax));
        const float f = to_2p15(e);
        float sum = (q[0] + q[1]) + (q[2] + q[3]);
#pragma unroll
        for (int d = 8; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
        if ((lane & 15) == 0) qhead[warp][lane >> 4] = sum;
        if (lane == 0) qhead[warp][2] = pow2_field(e - 14);  // 1 / f
        const int unit = (lane & 15) >> 1, w = (lane >> 4) + 2 * (unit & 1);
        __half* hi = reinterpret_cast<__half*>(&frag[0][w][0][4 * warp + (unit >> 1)]) + (lane & 1);
        __half* lo = reinterpret_cast<__half*>(&frag[kParts - 1][w][0][4 * (kPack ? warp + 4 : warp) + (unit >> 1)]) + (lane & 1);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float v = (j & 1 ? 0.0625f * q[j] : q[j] - 0.0625f * q[j + 1]) * f;
            const __half h = __float2half_rn(v);
            const int at = (j >> 1) * (32 * 4) + (j & 1) * 2;
            hi[at] = h;
            lo[at] = __float2half_rn(v - __half2float(h));
        }
    }
    // the new row: rounded to bf16, quantised, written to the cache, and kept as
    // the cache holds it.  Only its own score waits for the queries, and nothing
    // waits for it before the merge: its key takes longer than a query.
    const auto store_new = [&](float v[4], uint8_t* codes, uint32_t* pars, int at_row, float4* keep) {
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = round_bf16(v[j]);
        uint32_t par;
        const uint32_t code = quant_row(v, &par);
        const bool writes = !(g & p.halves);  // one of two that share the row
        if (writes) store_row(code, par, codes + (base + p.pos) * kRowBytes, pars + (base + p.pos) * 2, lane);
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = fmaf(bf16lo(par), (float)((code >> (4 * j)) & 15u), bf16hi(par));
        const float4 q = make_float4(v[0], v[1], v[2], v[3]);
        if (keep) keep[lane] = q;
        if (p.kv_row && writes) reinterpret_cast<float4*>(p.kv_row)[(size_t)at_row * (kHeadDim / 4) + lane] = q;
    };
    constexpr int kThreads = kAttnWarps * 32;
    if (new_k) {
        asm volatile("bar.arrive 1, %0;" ::"n"(kThreads) : "memory");
        float k[4];
        norm_rope_exact(x, gain, rope, p.eps, lane, k);
        store_new(k, p.k4, p.k_par, kv, nullptr);
        asm volatile("bar.sync 2, %0;" ::"n"(kThreads) : "memory");
        // the new position is a partial of its own: weight 1 at its score
#pragma unroll
        for (int j = 0; j < G; ++j) {
            const float4 q = reinterpret_cast<const float4*>(qs[j])[lane];
            const float s = warp_sum(fmaf(q.x, k[0], fmaf(q.y, k[1], fmaf(q.z, k[2], q.w * k[3]))));
            if (lane == 0) {
                wm[kAttnWarps][j] = s;
                wl[kAttnWarps][j] = 1.f;
            }
        }
    } else {
        if (new_v) {
            float v[4] = {x.x, x.y, x.z, x.w};
            store_new(v, p.v4, p.v_par, p.n_kv + kv, reinterpret_cast<float4*>(vnew));
        }
        asm volatile("bar.sync 1, %0;" ::"n"(kThreads) : "memory");
        if (has_new) asm volatile("bar.arrive 2, %0;" ::"n"(kThreads) : "memory");
    }

    // lane (r, t): positions r and r + 8 of a tile, query heads hd and hd + 1
    // (packed: lanes t and t ^ 2 share them, one with the high parts' columns
    // and one with the low parts')
    const int hd = kPack ? 2 * (t & 1) : 2 * t;
    uint2 qb[kParts][4][2];
    {
        const bool used = !kPack || (r & 3) < G;
#pragma unroll
        for (int q = 0; q < kParts; ++q)
#pragma unroll
            for (int w = 0; w < 4; ++w)
#pragma unroll
                for (int i = 0; i < 2; ++i) qb[q][w][i] = used ? frag[q][w][i][lane] : make_uint2(0, 0);
    }
    float qsum[2][2], fq[2];
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        const bool used = hd + c < G;
        qsum[0][c] = used ? qhead[hd + c][0] : 0.f;
        qsum[1][c] = used ? qhead[hd + c][1] : 0.f;
        fq[c] = used ? qhead[hd + c][2] : 0.f;
    }

    // M: the maximum the weights are relative to (it may lag the true one by
    // up to 8, a factor 256, and is then moved for all lanes of a warp);
    // fv[h]: the power of two that keeps |weight x V scale| of half h under
    // 2^15; both per head.  l and omin are this lane's positions' shares.
    float M[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f}, fv[2][2], omin[2][2] = {};
    fv[0][0] = fv[0][1] = fv[1][0] = fv[1][1] = to_2p9(15);
    float o[2][4][4];  // [half][16-channel block][row r: heads, row r + 8: heads]
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int c = 0; c < 4; ++c) o[h][i][c] = 0.f;

    const uint8_t* kst = my_ring + r * kRowBytes + t * 16;
    const uint8_t* vst = my_ring + kStageV + (r >> 2) * 128 + (2 * t + ((r >> 1) & 1)) * 16 + (r & 1) * 8;
    const uint8_t* pst = my_ring + kStagePar + r * 8;
    float sc[2][2];  // [position][head]
    auto scores = [&](int so) {
        const uint4 wa = *reinterpret_cast<const uint4*>(kst + so);
        const uint4 wb = *reinterpret_cast<const uint4*>(kst + so + 8 * kRowBytes);
        const uint2 par[2] = {*reinterpret_cast<const uint2*>(pst + so), *reinterpret_cast<const uint2*>(pst + so + 64)};
        const uint32_t w[2][4] = {{wa.x, wa.y, wa.z, wa.w}, {wb.x, wb.y, wb.z, wb.w}};
        float c[2][4];
#pragma unroll
        for (int i = 0; i < 4; i += 2)
#pragma unroll
            for (int s = 0; s < 2; ++s)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint32_t u = nibble_bytes(w[0][i + h], s), v = nibble_bytes(w[1][i + h], s);
                    const uint32_t a[4] = {low_code(u), low_code(v), both_codes(u), both_codes(v)};
                    if (i == 0 && s == 0)
                        mma16816_first(c[h], a, qb[0][i + h][s]);
                    else
                        mma16816(c[h], a, qb[0][i + h][s]);
                    if (!kPack) mma16816(c[h], a, qb[kParts - 1][i + h][s]);
                }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const float centre0 = fmaf(8.f, bf16lo(par[k].x), bf16hi(par[k].x));
            const float centre1 = fmaf(8.f, bf16lo(par[k].y), bf16hi(par[k].y));
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                float x = fmaf(c[1][2 * k + j], bf16lo(par[k].y), c[0][2 * k + j] * bf16lo(par[k].x));
                if (kPack) x += __shfl_xor_sync(0xffffffffu, x, 2);
                sc[k][j] = fmaf(x, fq[j], fmaf(centre0, qsum[0][j], centre1 * qsum[1][j]));
            }
        }
    };
    float wf[2][2][2];  // [half][position][head]
    // V codes are centred at 8 at even positions (a register's low half) and at 7 at
    // odd ones, 7.5 on average, the middle of a half's range
    constexpr uint32_t kLowV = 0x64076408u, kBothV = 0x64776488u;
    const float centre_v = r & 1 ? 7.f : 8.f;
    auto output = [&](int so) {
        uint2 vw[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) vw[i] = *reinterpret_cast<const uint2*>(vst + so + i * 256);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            uint32_t hi[2], lo[2];
            split_h2(wf[h][0][0], wf[h][0][1], &hi[0], &lo[0]);
            split_h2(wf[h][1][0], wf[h][1][1], &hi[1], &lo[1]);
            uint2 b[kParts];
            if (kPack) {
                b[0] = make_uint2(transpose8(t < 2 ? hi[0] : lo[0]), transpose8(t < 2 ? hi[1] : lo[1]));
            } else {
                b[0] = make_uint2(transpose8(hi[0]), transpose8(hi[1]));
                b[kParts - 1] = make_uint2(transpose8(lo[0]), transpose8(lo[1]));
            }
            const uint32_t w0 = h ? vw[0].y : vw[0].x, w1 = h ? vw[1].y : vw[1].x;
            const uint32_t w2 = h ? vw[2].y : vw[2].x, w3 = h ? vw[3].y : vw[3].x;
            // block i: rows r are nibble 2 i of word r (channel 64 h + 8 r + 2 i),
            // rows r + 8 that and 16 times nibble 2 i + 1
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t sel = i < 2 ? 0x5410u : 0x7632u;
                const uint32_t x = nibble_bytes(__byte_perm(w0, w1, sel), i & 1);
                const uint32_t y = nibble_bytes(__byte_perm(w2, w3, sel), i & 1);
                const uint32_t a[4] = {low_code(x, kLowV), both_codes(x, kBothV), low_code(y, kLowV), both_codes(y, kBothV)};
                mma16816(o[h][i], a, b[0]);
                if (!kPack) mma16816(o[h][i], a, b[kParts - 1]);
            }
        }
    };

    int stage = 0, tile = split * p.tiles_per_split + warp;
    if (tile < tile_end) {
        cp_async_wait<kStages - 2>();
        __syncwarp();
        scores(0);
    }
    for (; tile < tile_end; tile += kAttnWarps) {
        __syncwarp();
        {
            int fill = stage + kStages - 1;
            if (fill >= kStages) fill -= kStages;
            if (next < tile_end) copy.issue(next, fill, lane);
            cp_async_commit();
            next += kAttnWarps;
        }
        const int so = stage * kStageBytes;
        if (++stage == kStages) stage = 0;

        if (tile * kTilePos + kTilePos > p.pos) {
            const int left = p.pos - tile * kTilePos - r;
#pragma unroll
            for (int k = 0; k < 2; ++k)
                if (8 * k >= left) sc[k][0] = sc[k][1] = -INFINITY;
        }
        float mx[2] = {fmaxf(sc[0][0], sc[1][0]), fmaxf(sc[0][1], sc[1][1])};
        if (__any_sync(0xffffffffu, mx[0] > M[0] + 8.f || mx[1] > M[1] + 8.f)) {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
#pragma unroll
                for (int d = 4; d <= 16; d <<= 1) mx[c] = fmaxf(mx[c], __shfl_xor_sync(0xffffffffu, mx[c], d));
                if (mx[c] > M[c]) {
                    const float corr = ex2(M[c] - mx[c]);
                    M[c] = mx[c];
                    l[c] *= corr;
                    // weights so far shrink by corr: so does what they are kept under
                    const int shrink = (int)(__float_as_uint(corr) >> 23) - 127;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int e_old = expo_of(fv[h][c]), e_new = max(e_old + shrink, 15);
                        const float k = corr * pow2_field(min(127 + e_old - e_new, 254));
                        fv[h][c] = to_2p9(e_new);
                        omin[h][c] *= corr;
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            o[h][i][c] *= k;
                            o[h][i][2 + c] *= k;
                        }
                    }
                }
            }
        }

        // ---- weights, and the same times each position's V scale
        {
            const uint2 par[2] = {*reinterpret_cast<const uint2*>(pst + so + 128),
                                  *reinterpret_cast<const uint2*>(pst + so + 192)};
            float wx = 0.f, vs[2][2][2];
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const float pw = ex2(sc[k][c] - M[c]);
                    l[c] += pw;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint32_t u = h ? par[k].y : par[k].x;
                        omin[h][c] = fmaf(pw, fmaf(centre_v, bf16lo(u), bf16hi(u)), omin[h][c]);
                        vs[h][k][c] = pw * bf16lo(u);
                        wf[h][k][c] = vs[h][k][c] * fv[h][c];
                        wx = fmaxf(wx, fabsf(wf[h][k][c]));
                    }
                }
            if (__any_sync(0xffffffffu, wx >= 32768.f)) {
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        float m = fmaxf(fabsf(vs[h][0][c]), fabsf(vs[h][1][c]));
#pragma unroll
                        for (int d = 4; d <= 16; d <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
                        const int e_old = expo_of(fv[h][c]), e_new = max(e_old, expo(m));
                        const float k = pow2_field(max(127 + e_old - e_new, 0));
                        fv[h][c] = to_2p9(e_new);
                        wf[h][0][c] = vs[h][0][c] * fv[h][c];
                        wf[h][1][c] = vs[h][1][c] * fv[h][c];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            o[h][i][c] *= k;
                            o[h][i][2 + c] *= k;
                        }
                    }
            }
        }
        // the output product of this tile beside the scores of the next: two
        // independent streams of tensor and integer work
        if (tile + kAttnWarps < tile_end) {
            cp_async_wait<kStages - 2>();
            __syncwarp();
            output(so);
            scores(stage * kStageBytes);
        } else {
            output(so);
        }
    }

    // ---- this warp's partial: maximum, sum, output (its ring is free now)
    cp_async_wait<0>();
    __syncwarp();
#pragma unroll
    for (int c = 0; c < 2; ++c) {
#pragma unroll
        for (int d = 4; d <= 16; d <<= 1) {
            l[c] += __shfl_xor_sync(0xffffffffu, l[c], d);
            omin[0][c] += __shfl_xor_sync(0xffffffffu, omin[0][c], d);
            omin[1][c] += __shfl_xor_sync(0xffffffffu, omin[1][c], d);
        }
        if (r == 0 && (!kPack || t < 2) && hd + c < G) {
            wm[warp][hd + c] = M[c];
            wl[warp][hd + c] = l[c];
        }
        float* po = reinterpret_cast<float*>(my_ring) + (hd + c) * kHeadDim + 8 * r;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float back = pow2_field(expo_of(fv[h][c]) - 8);  // 1 / fv
            float v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                float x = i & 1 ? o[h][i >> 1][2 + c] - o[h][i >> 1][c] : o[h][i >> 1][c];
                if (kPack) x += __shfl_xor_sync(0xffffffffu, x, 2);
                v[i] = fmaf(i & 1 ? x * 0.0625f : x, back, omin[h][c]);
            }
            if ((!kPack || t < 2) && hd + c < G) {
                reinterpret_cast<float4*>(po + 64 * h)[0] = make_float4(v[0], v[1], v[2], v[3]);
                reinterpret_cast<float4*>(po + 64 * h)[1] = make_float4(v[4], v[5], v[6], v[7]);
            }
        }
    }
    __syncthreads();
    // all blocks of the cluster run: their shared memory may be written
    if (p.cluster) asm volatile("barrier.cluster.wait.aligned;" ::: "memory");

    // ---- merge the warps and the new row, in order.  A partial with sum 0 is
    // empty; NaN sums pass through.
    const int parts = has_new ? kAttnWarps + 1 : kAttnWarps;
    const size_t unit = (size_t)g * p.S + split;
    if (warp < G) {
        const bool in = lane < parts;
        const float pm = in ? wm[lane][warp] : -INFINITY, pl = in ? wl[lane][warp] : 0.f;
        const float mx = warp_max(pm);
        const float c = pl == 0.f ? 0.f : ex2(pm - mx);
        const float L = warp_sum(pl == 0.f ? 0.f : pl * c);
        if (in) merge_c[lane][warp] = c;
        if (lane == 0) {
            merge_l[warp] = L;
            if (p.S > 1 && !p.cluster) p.part_ml[unit * G + warp] = make_float2(mx, L);
        }
        if (p.cluster && lane < p.S) store_remote(&box_ml[split][warp], lane, make_float2(mx, L));
    }
    __syncthreads();
    constexpr int kVec = G * kHeadDim / 4;  // the group's outputs, four a thread
    const int share = p.cluster ? (kVec + p.S - 1) / p.S : kVec;
    if (threadIdx.x < kVec) {
        const int j = threadIdx.x / (kHeadDim / 4), d4 = threadIdx.x % (kHeadDim / 4);
        float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w <= kAttnWarps; ++w) {
            if (w >= parts || wl[w][j] == 0.f) continue;  // an empty warp's ring holds no output
            const float c = merge_c[w][j];
            const float4 v = w < kAttnWarps ? reinterpret_cast<const float4*>(ring + w * kRingBytes)[threadIdx.x]
                                            : reinterpret_cast<const float4*>(vnew)[d4];
            O.x = fmaf(v.x, c, O.x);
            O.y = fmaf(v.y, c, O.y);
            O.z = fmaf(v.z, c, O.z);
            O.w = fmaf(v.w, c, O.w);
        }
        if (p.S == 1) {
            const float L = merge_l[j];
            reinterpret_cast<float4*>(p.out)[(size_t)g * kVec + threadIdx.x] = make_float4(O.x / L, O.y / L, O.z / L, O.w / L);
        } else if (p.cluster) {
            const int to = threadIdx.x / share;
            store_remote(&box_o[split * share + threadIdx.x - to * share], to, O);
        } else {
            reinterpret_cast<float4*>(p.part_o)[unit * kVec + threadIdx.x] = O;
        }
    }
    if (p.S == 1) return;

    // ---- a cluster: each block joins its share of the outputs, in order
    if (p.cluster) {
        asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
        asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
        const int vec = split * share + threadIdx.x;
        if (threadIdx.x < share && vec < kVec) {
            const int j = vec / (kHeadDim / 4);
            float mx = -INFINITY, L = 0.f;
            for (int s = 0; s < p.S; ++s) mx = fmaxf(mx, box_ml[s][j].x);
            float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int s = 0; s < p.S; ++s) {
                const float2 ml = box_ml[s][j];
                const float4 v = box_o[s * share + threadIdx.x];
                const float c = ex2(ml.x - mx);
                L = fmaf(ml.y, c, L);
                O.x = fmaf(v.x, c, O.x);
                O.y = fmaf(v.y, c, O.y);
                O.z = fmaf(v.z, c, O.z);
                O.w = fmaf(v.w, c, O.w);
            }
            reinterpret_cast<float4*>(p.out)[(size_t)g * kVec + vec] = make_float4(O.x / L, O.y / L, O.z / L, O.w / L);
        }
        return;
    }

    // ---- the last split of this kv head to finish merges all splits, in order
    __syncthreads();
    if (threadIdx.x == 0) {
        // releases the block's partials (ordered before it by the barrier) and,
        // for the last, acquires the others'
        unsigned ticket;
        asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;" : "=r"(ticket) : "l"(&p.tickets[g]) : "memory");
        s_last = ticket == (unsigned)(p.S - 1);
    }
    __syncthreads();
    if (!s_last) return;
    // thread (part, vector): every kTeams-th split, all its first loads in flight
    // while the weights are found
    constexpr int kTeams = kAttnWarps * 32 / kVec;
    constexpr int kAhead = 8;
    const int part = threadIdx.x / kVec, vec = threadIdx.x % kVec, head = vec / (kHeadDim / 4);
    const float4* po = reinterpret_cast<const float4*>(p.part_o) + (size_t)g * p.S * kVec + vec;
    float4 ahead[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
        const int s = part + i * kTeams;
        ahead[i] = part < kTeams && s < p.S ? __ldcg(po + (size_t)s * kVec) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    if (warp < G) {
        const float2* ml = p.part_ml + (size_t)g * p.S * G + warp;
        constexpr int kMost = (kMaxSplitUnits + 31) / 32;
        float2 v[kMost];
        float mx = -INFINITY;
#pragma unroll
        for (int i = 0; i < kMost; ++i) {
            v[i] = lane + 32 * i < p.S ? __ldcg(ml + (size_t)(lane + 32 * i) * G) : make_float2(-INFINITY, 0.f);
            mx = fmaxf(mx, v[i].x);
        }
        mx = warp_max(mx);
        float L = 0.f;
#pragma unroll
        for (int i = 0; i < kMost; ++i)
            if (lane + 32 * i < p.S) {
                const float c = ex2(v[i].x - mx);
                merge_c[lane + 32 * i][warp] = c;
                L = fmaf(v[i].y, c, L);
            }
        L = warp_sum(L);
        if (lane == 0) merge_l[warp] = L;
    }
    __syncthreads();
    float4* parts_o = reinterpret_cast<float4*>(ring);  // [kTeams][kVec]
    if (part < kTeams) {
        float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int s0 = part; s0 < p.S; s0 += kAhead * kTeams) {
            if (s0 != part) {
#pragma unroll
                for (int i = 0; i < kAhead; ++i) {
                    const int s = s0 + i * kTeams;
                    if (s < p.S) ahead[i] = __ldcg(po + (size_t)s * kVec);
                }
            }
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                const int s = s0 + i * kTeams;
                if (s >= p.S) break;
                const float c = merge_c[s][head];
                O.x = fmaf(ahead[i].x, c, O.x);
                O.y = fmaf(ahead[i].y, c, O.y);
                O.z = fmaf(ahead[i].z, c, O.z);
                O.w = fmaf(ahead[i].w, c, O.w);
            }
        }
        parts_o[threadIdx.x] = O;
    }
    __syncthreads();
    if (threadIdx.x < kVec) {
        float4 O = parts_o[threadIdx.x];
#pragma unroll
        for (int q = 1; q < kTeams; ++q) {
            const float4 v = parts_o[q * kVec + threadIdx.x];
            O.x += v.x;
            O.y += v.y;
            O.z += v.z;
            O.w += v.w;
        }
        const float L = merge_l[head];
        reinterpret_cast<float4*>(p.out)[(size_t)g * kVec + threadIdx.x] = make_float4(O.x / L, O.y / L, O.z / L, O.w / L);
    }
    if (threadIdx.x == 0) p.tickets[g] = 0u;
}

int max_splits(int n_kv) { return n_kv >= kMaxSplitUnits ? 1 : kMaxSplitUnits / n_kv; }

// How many clusters of c blocks run at once.
struct Room {
    int clusters[kMaxCluster + 1];
    // the most blocks a cluster may have for `heads` clusters to run at once
    int most(int heads) const {
        int c = kMaxCluster;
        while (c > 1 && clusters[c] < heads) --c;
        return c;
    }
};

// Per device: the shared-memory limit raised, and the clusters there is room for (a
// cluster stays within a group of SMs; above 8 blocks is this device's own, so it is
// asked for).
template <int G>
cudaError_t prepare_attn_kv4(int dev, int sms, Room* room) {
    static std::mutex mu;
    static Room rooms[64] = {};
    const auto kern = attn_kv4_kernel<G>;
    const std::lock_guard<std::mutex> lock(mu);
    Room& known = rooms[dev & 63];
    if (!known.clusters[1]) {
        cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kAttnSmem);
        if (e != cudaSuccess) return e;
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return e;
        Room r = {{0, sms}};
        for (int c = 2; c <= kMaxCluster; ++c) {
            e = clusters_at_once(kern, kAttnWarps * 32, kAttnSmem, c, 1, &r.clusters[c]);
            if (e != cudaSuccess) return e;
        }
        known = r;
    }
    *room = known;
    return cudaSuccess;
}

template <int G>
cudaError_t launch_attn_kv4(Kv4Params p, int dev, int sms, cudaStream_t s) {
    Room room;
    const cudaError_t e = prepare_attn_kv4<G>(dev, sms, &room);
    if (e != cudaSuccess) return e;
    const int tiles = (p.pos + kTilePos - 1) / kTilePos;
    if constexpr (G >= 4) {
        // The queries of a head as two heads, which read the cache twice, while SMs are
        // left.  Eight as four and four: a tile takes a warp a sixth less time and a
        // call 1 us less for its queries and partials (16/2 heads, 1000 positions 5.1 us
        // against 5.9, 20000 9.8 against 11.6), while that leaves a warp one tile, or
        // four where there are SMs for sixteen blocks a head (64/8 heads, 6000
        // positions 9.7 against 9.1; 32/4, 40000 16.6 against 15.0).  Four as two and two
        // save 0.3 us while half the warps have a tile (32/8 heads, position 0 3.7 against
        // 4.0, 700 5.1 against 5.6, but 1279 5.8 against 5.5).
        const int heads = 2 * p.n_kv, wide = sms / heads, turn = kAttnWarps * room.most(heads);
        const bool two = G == 8 ? tiles <= turn || (wide >= 16 && tiles <= 4 * kAttnWarps * wide) : tiles <= turn / 2;
        if (two && wide >= 1 && !p.halves) {
            p.halves = 1;
            return launch_attn_kv4<G / 2>(p, dev, sms, s);
        }
    }
    // How a head's cache is split, none empty (us a call at 32/8 heads, none of
    // them as two):
    // - up to 192 positions one block takes it: 4.3 at 100 against 5.0 in two
    //   blocks, 5.05 at 200 against 4.9 in four;
    // - then a cluster, whose blocks join through shared memory, four tiles a
    //   block up to the largest cluster that all heads find room for at once: 5.1 at
    //   300 (one block 5.6, blocks of eight tiles 5.2), 5.5 at 1280 (joined through
    //   global memory 7.4, blocks of 16 tiles in clusters of at most eight 6.6);
    // - and where that leaves a warp more than two tiles, blocks all over the
    //   device, a tile a warp, joined through global memory: 8.5 at 8000
    //   positions against 8.7, but 7.8 at 5000 against 7.5.  Eight queries a head, with
    //   partials twice as large, break even at three tiles.
    const int heads = p.n_kv << p.halves;
    int S = 1;
    if (tiles > kOneBlockTiles) {
        S = std::min(room.most(heads), (tiles + kClusterTiles - 1) / kClusterTiles);
        p.cluster = S > 1 && tiles <= S * kAttnWarps * (G == 8 ? 3 : 2);
        if (!p.cluster)
            S = std::max(1, std::min({(tiles + kAttnWarps - 1) / kAttnWarps, max_splits(p.n_kv), sms / heads}));
    }
    p.tiles_per_split = std::max(1, (tiles + S - 1) / S);
    p.S = std::max(1, (tiles + p.tiles_per_split - 1) / p.tiles_per_split);
    return launch_ordered(attn_kv4_kernel<G>, dim3(heads, p.S), dim3(kAttnWarps * 32), kAttnSmem, s, p.cluster ? p.S : 1, 1, p);
}

bool misaligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0; }

int report_kv4(cudaError_t e, const char* what) {
    std::fprintf(stderr, "tts: %s failed: %s\n", what, cudaGetErrorString(e));
    return TTS_ERR_CUDA;
}


// [tickets][outputs: 128 words per split and query head][maximum and sum: 2
// words per split and query head].  The tickets' place does not depend on the
// heads, so a workspace may serve calls of different shapes in turn.
size_t workspace_bytes_for(int n_q, int n_kv) {
    return kTicketBytes + (size_t)n_q * max_splits(n_kv) * (2 + kHeadDim) * 4;
}

bool heads_ok(int n_q, int n_kv) {
    if (n_kv < 1 || n_kv > kKv4MaxKvHeads || n_q < 1 || n_q > kKv4MaxHeads || n_q % n_kv) return false;
    const int G = n_q / n_kv;
    return G == 1 || G == 2 || G == 4 || G == 8;
}

// in: the 4-bit cache is written, else the bf16 ones.
int rows_ok(bool in, const void* k, const void* v, const void* k4, const void* v4, const void* kp, const void* vp,
            int n_kv, int p0, int p1, int stride, int max_pos) {
    if (!k || !v || !k4 || !v4 || !kp || !vp || n_kv < 1 || n_kv > kKv4MaxKvHeads) return TTS_ERR_ARG;
    if (max_pos < 1 || max_pos > kKv4MaxPos || p0 < 0 || p1 < p0) return TTS_ERR_ARG;
    if (misaligned(k, 16) || misaligned(v, 16) || misaligned(k4, 16) || misaligned(v4, 16) || misaligned(kp, 16) ||
        misaligned(vp, 16))
        return TTS_ERR_ARG;
    if (p1 > max_pos) return TTS_ERR_FULL;
    if (p1 > stride) return TTS_ERR_ARG;
    const size_t rows = (size_t)n_kv * max_pos, bytes = (size_t)n_kv * stride * kHeadDim * 2;
    const Span wide[] = {{k, bytes}, {v, bytes}};
    const Span packed[] = {{k4, rows * kRowBytes}, {v4, rows * kRowBytes}, {kp, rows * 8}, {vp, rows * 8}};
    if (in ? overwritten(packed, wide) : overwritten(wide, packed)) return TTS_ERR_ARG;
    return TTS_OK;
}

}  // namespace
}  // namespace tts

extern "C" int tts_quantize_kv4(const void* k, const void* v, int n_kv, int p0, int p1, int src_stride, void* k4,
                                void* v4, void* k_par, void* v_par, int max_pos, void* stream) {
    using namespace tts;
    const int rc = rows_ok(true, k, v, k4, v4, k_par, v_par, n_kv, p0, p1, src_stride, max_pos);
    if (rc != TTS_OK || p0 == p1) return rc;
    const RowParams p{static_cast<const uint8_t*>(k4),      static_cast<const uint8_t*>(v4),
                      static_cast<const uint32_t*>(k_par),  static_cast<const uint32_t*>(v_par),
                      static_cast<const uint16_t*>(k),      static_cast<const uint16_t*>(v),
                      p0, p1 - p0, src_stride, max_pos};
    const cudaError_t e = launch_ordered(quantize_kv4_kernel, dim3((p.np + kBlockRows - 1) / kBlockRows, 2 * n_kv),
                                         dim3(kRowThreads), 0, static_cast<cudaStream_t>(stream), 1, 1, p);
    return e == cudaSuccess ? TTS_OK : report_kv4(e, "tts_quantize_kv4");
}

extern "C" int tts_dequantize_kv4(const void* k4, const void* v4, const void* k_par, const void* v_par, int n_kv,
                                  int p0, int p1, int max_pos, void* k, void* v, int dst_stride, void* stream) {
    using namespace tts;
    const int rc = rows_ok(false, k, v, k4, v4, k_par, v_par, n_kv, p0, p1, dst_stride, max_pos);
    if (rc != TTS_OK || p0 == p1) return rc;
    const RowParams p{static_cast<const uint8_t*>(k4),      static_cast<const uint8_t*>(v4),
                      static_cast<const uint32_t*>(k_par),  static_cast<const uint32_t*>(v_par),
                      static_cast<const uint16_t*>(k),      static_cast<const uint16_t*>(v),
                      p0, p1 - p0, dst_stride, max_pos};
    const cudaError_t e = launch_ordered(dequantize_kv4_kernel, dim3((p.np + kBlockRows - 1) / kBlockRows, 2 * n_kv),
                                         dim3(kRowThreads), 0, static_cast<cudaStream_t>(stream), 1, 1, p);
    return e == cudaSuccess ? TTS_OK : report_kv4(e, "tts_dequantize_kv4");
}

extern "C" int tts_attention_kv4_workspace(int n_q, int n_kv, size_t* bytes) {
    using namespace tts;
    if (!bytes || !heads_ok(n_q, n_kv)) return TTS_ERR_ARG;
    *bytes = workspace_bytes_for(n_q, n_kv);
    return TTS_OK;
}

extern "C" int tts_attention_decode_kv4(const float* qkv, const void* q_norm, const void* k_norm, void* k4, void* v4,
                                        void* k_par, void* v_par, float* out, float* kv_row, int n_q, int n_kv,
                                        int max_pos, int pos, float eps, float rope_theta, void* workspace,
                                        size_t workspace_bytes, void* stream) {
    using namespace tts;
    if (!qkv || !q_norm || !k_norm || !k4 || !v4 || !k_par || !v_par || !out || !workspace) return TTS_ERR_ARG;
    if (!heads_ok(n_q, n_kv) || max_pos < 1 || max_pos > kKv4MaxPos || pos < 0) return TTS_ERR_ARG;
    if (!(eps >= 0.f) || !(rope_theta > 0.f) || !std::isfinite(rope_theta)) return TTS_ERR_ARG;
    if (misaligned(qkv, 16) || misaligned(q_norm, 16) || misaligned(k_norm, 16) || misaligned(k4, 16) ||
        misaligned(v4, 16) || misaligned(k_par, 16) || misaligned(v_par, 16) || misaligned(out, 16) ||
        misaligned(kv_row, 16) || misaligned(workspace, 16))
        return TTS_ERR_ARG;
    if (workspace_bytes < workspace_bytes_for(n_q, n_kv)) return TTS_ERR_ARG;
    {
        const size_t head = sizeof(float) * kHeadDim, rows = (size_t)n_kv * max_pos;
        if (overwritten({{out, n_q * head},
                         {kv_row, 2 * n_kv * head},
                         {k4, rows * kRowBytes},
                         {v4, rows * kRowBytes},
                         {k_par, rows * 8},
                         {v_par, rows * 8},
                         {workspace, workspace_bytes_for(n_q, n_kv)}},
                        {{qkv, (n_q + 2 * n_kv) * head}, {q_norm, 2 * kHeadDim}, {k_norm, 2 * kHeadDim}}))
            return TTS_ERR_ARG;
    }
    if (pos >= max_pos) return TTS_ERR_FULL;
    Kv4Params p{};
    p.qkv = qkv;
    p.q_norm = static_cast<const __nv_bfloat16*>(q_norm);
    p.k_norm = static_cast<const __nv_bfloat16*>(k_norm);
    p.k4 = static_cast<uint8_t*>(k4);
    p.v4 = static_cast<uint8_t*>(v4);
    p.k_par = static_cast<uint32_t*>(k_par);
    p.v_par = static_cast<uint32_t*>(v_par);
    p.out = out;
    p.kv_row = kv_row;
    p.n_q = n_q;
    p.n_kv = n_kv;
    p.max_pos = max_pos;
    p.pos = pos;
    p.eps = eps;
    // theta^(-i/64) from its square roots' products (a few ulp of fp64; 64 calls of
    // pow would take longer than the launch)
    double freq[kHeadDim / 2];
    freq[0] = 1.0;
    freq[1] = std::pow((double)rope_theta, -2.0 / (double)kHeadDim);
    for (int i = 2; i < kHeadDim / 2; ++i) freq[i] = freq[i / 2] * freq[i - i / 2];
    for (int i = 0; i < kHeadDim / 2; ++i) {
        double c, sn;
        sincos((double)pos * freq[i], &sn, &c);
        p.rope.cs[i] = make_float2((float)c, (float)sn);
        p.rope.rest[i] = make_float2((float)(c - (double)(float)c), (float)(sn - (double)(float)sn));
    }
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return TTS_ERR_CUDA;
    char* ws = static_cast<char*>(workspace);
    p.tickets = reinterpret_cast<unsigned*>(ws);
    p.part_o = reinterpret_cast<float*>(ws + kTicketBytes);  // 16-byte vectors: before the 8-byte ones
    p.part_ml = reinterpret_cast<float2*>(p.part_o + (size_t)n_q * max_splits(n_kv) * kHeadDim);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    switch (n_q / n_kv) {
        case 1: e = launch_attn_kv4<1>(p, dev, sms, st); break;
        case 2: e = launch_attn_kv4<2>(p, dev, sms, st); break;
        case 4: e = launch_attn_kv4<4>(p, dev, sms, st); break;
        default: e = launch_attn_kv4<8>(p, dev, sms, st); break;
    }
    return e == cudaSuccess ? TTS_OK : report_kv4(e, "tts_attention_decode_kv4");
}
