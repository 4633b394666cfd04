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
#include <atomic>
#include <cmath>
#include <cstdio>

#include "kernels.h"
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
__device__ __forceinline__ void rope_at(const RopeRow& r, int i, float* c, float* s) {
    const float2 v = r.cs[i];
    *c = v.x;
    *s = v.y;
}
__device__ __forceinline__ void rope_at(const RopeRow& r, int i, double* c, double* s) {
    const float2 v = r.cs[i], d = r.rest[i];
    *c = (double)v.x + (double)d.x;
    *s = (double)v.y + (double)d.y;
}

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
    unsigned* tickets;       // [n_kv], zero between calls
    float2* part_ml;         // [n_kv][S][G] maximum, sum
    float* part_o;           // [n_kv][S][G][128]
    RopeRow rope;
};

// Quantise one row held by a warp: lane l has channels 4l .. 4l + 3 (bf16
// values), so lanes 0-15 hold half 0 and lanes 16-31 half 1.  Returns the
// lane's four codes in 16 bits; *par is its half's parameter word.  The
// arithmetic is IEEE fp32 as defined above.  A half whose range is not finite
// (it holds a NaN or an infinity) gets NaN parameters: its values read as NaN.
__device__ __forceinline__ uint32_t quant_row(const float x[4], uint32_t* par) {
    float lo = fminf(fminf(x[0], x[1]), fminf(x[2], x[3]));
    float hi = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
    int bad = !(isfinite(x[0]) && isfinite(x[1]) && isfinite(x[2]) && isfinite(x[3]));
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) {
        lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
        hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
        bad |= __shfl_xor_sync(0xffffffffu, bad, o);
    }
    const __nv_bfloat16 sb = __float2bfloat16_rn(__fdiv_rn(hi - lo, 15.f));
    const float s = __bfloat162float(sb);
    if (bad || !isfinite(s)) {
        *par = 0x7fff7fffu;
        return 0;
    }
    uint32_t code = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float q = s > 0.f ? fminf(fmaxf(rintf(__fdiv_rn(x[j] - lo, s)), 0.f), 15.f) : 0.f;
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
// Lane l's four values of a cached row.
__device__ __forceinline__ void load_row(const uint8_t* row, const uint32_t* par_row, int lane, float v[4]) {
    const uint32_t code = *reinterpret_cast<const uint16_t*>(row + lane_byte(lane));
    const uint32_t par = par_row[lane >> 4];
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = fmaf(bf16lo(par), (float)((code >> (4 * j)) & 15u), bf16hi(par));
}

__global__ void __launch_bounds__(256) quantize_kv4_kernel(const uint16_t* k, const uint16_t* v, int n_kv, int p0,
                                                           int np, int src_stride, uint8_t* k4, uint8_t* v4,
                                                           uint32_t* k_par, uint32_t* v_par, int max_pos) {
    const int lane = threadIdx.x & 31;
    const int i = blockIdx.x * 8 + (threadIdx.x >> 5);
    if (i >= np) return;
    const int head = blockIdx.y >> 1;
    const bool is_v = blockIdx.y & 1;
    const uint16_t* src = (is_v ? v : k) + ((size_t)head * src_stride + p0 + i) * kHeadDim + 4 * lane;
    const uint2 w = *reinterpret_cast<const uint2*>(src);
    const float x[4] = {bf16lo(w.x), bf16hi(w.x), bf16lo(w.y), bf16hi(w.y)};
    uint32_t par;
    const uint32_t code = quant_row(x, &par);
    const size_t at = (size_t)head * max_pos + p0 + i;
    store_row(code, par, (is_v ? v4 : k4) + at * kRowBytes, (is_v ? v_par : k_par) + at * 2, lane);
}

__global__ void __launch_bounds__(256) dequantize_kv4_kernel(const uint8_t* k4, const uint8_t* v4,
                                                             const uint32_t* k_par, const uint32_t* v_par, int n_kv,
                                                             int p0, int np, int max_pos, uint16_t* k, uint16_t* v,
                                                             int dst_stride) {
    const int lane = threadIdx.x & 31;
    const int i = blockIdx.x * 8 + (threadIdx.x >> 5);
    if (i >= np) return;
    const int head = blockIdx.y >> 1;
    const bool is_v = blockIdx.y & 1;
    const size_t at = (size_t)head * max_pos + p0 + i;
    float x[4];
    load_row((is_v ? v4 : k4) + at * kRowBytes, (is_v ? v_par : k_par) + at * 2, lane, x);
    uint16_t* dst = (is_v ? v : k) + ((size_t)head * dst_stride + p0 + i) * kHeadDim + 4 * lane;
#pragma unroll
    for (int j = 0; j < 4; ++j) dst[j] = __bfloat16_as_ushort(__float2bfloat16_rn(x[j]));
}

// q/k RMSNorm over the head then rotate-half RoPE, in type T: lane l has
// channels 4l .. 4l + 3, whose rotation partners sit in lane l ^ 16.
template <typename T>
__device__ __forceinline__ void norm_rope(const float* src, const __nv_bfloat16* gain, const RopeRow& rope, float eps,
                                          int lane, T o[4]) {
    T a[4], ss = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        a[j] = (T)src[4 * lane + j];
        ss += a[j] * a[j];
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, d);
    const T r = (T)1 / sqrt(ss / (T)kHeadDim + (T)eps);
#pragma unroll
    for (int j = 0; j < 4; ++j) a[j] = a[j] * r * (T)__bfloat162float(gain[4 * lane + j]);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const T partner = __shfl_xor_sync(0xffffffffu, a[j], 16);
        const int i = (4 * lane + j) & 63;
        T c, s;
        rope_at(rope, i, &c, &s);
        o[j] = lane < 16 ? a[j] * c - partner * s : a[j] * c + partner * s;
    }
}

// ---- the attention kernel -------------------------------------------------------
// A block takes one kv head and one contiguous range of 16-position tiles (a
// split); its warps take the range's tiles in turn, each with its own ring of
// asynchronous copies, running maximum, sum and output, so nothing in the loop
// waits for another warp.
//
// Both products run on the tensor cores (m16n8k16, fp16 operands, fp32 sums),
// with the codes as they lie in memory: a nibble masked out of its 16-bit half
// IS the fp16 subnormal u 2^-24 (or, from bits 4-7, 16 u 2^-24), exact, so a
// code costs 5/8 of an instruction and no conversion.  The powers of two and
// the factor 16 are taken back on the other operand or in the epilogue.
//   scores  A = queries (rows 0-7: the group's heads, fp16 high parts; rows
//           8-15: their low parts), B = K codes.  score = sum over halves of
//           s_K (q . u) + m_K sum(q): the scale and the minimum of a position
//           enter in fp32 on the accumulators.
//   output  A = weights p s_V of each position, again high and low parts in
//           rows r and r + 8, B = V codes; sum of p m_V beside it in fp32.
// Two fp16 parts of a value scaled by a power of two to below 2^15 keep 22
// bits (and 2^-39 of the row's largest), so nothing falls under fp32 accuracy
// by more than rounding of the sums.  The scaling of the weights follows their
// running maximum per head and half, like the softmax maximum.
//
// Column n of block b of a tile's 16 positions is position
// 4 (n / 2) + 2 b + n % 2: an accumulator's two columns and the two blocks of
// a lane are then four neighbouring positions, the ones whose V rows the lane
// reads, and the score accumulators are the weight operand without a shuffle.
constexpr int kAttnWarps = 12;
constexpr int kTilePos = 16;
constexpr int kStages = 6;
constexpr int kStageV = kTilePos * kRowBytes;             // K rows, then V rows (permuted)
constexpr int kStagePar = 2 * kStageV;                    // then K and V parameters
constexpr int kStageBytes = kStagePar + 2 * kTilePos * 8;
constexpr int kRingBytes = kStages * kStageBytes;         // per warp
constexpr int kAttnSmem = kAttnWarps * kRingBytes;
static_assert(kRingBytes >= 8 * kHeadDim * 4, "a warp's output partial reuses its ring");

__device__ __forceinline__ void cp_async16_zfill(uint32_t dst, const void* src, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async8_zfill(uint32_t dst, const void* src, int bytes) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ void mma16816(float c[4], const uint32_t a[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
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
// The biased exponent of w >= 0, at least 14, and the power of two that takes
// w to [2^14, 2^15).
__device__ __forceinline__ int expo(float w) { return max((int)(__float_as_uint(w) >> 23), 14); }
__device__ __forceinline__ float pow2_field(int field) { return __uint_as_float((uint32_t)field << 23); }
__device__ __forceinline__ float to_2p15(int e) { return pow2_field(268 - e); }

// Copies of one tile into a stage: codes of both caches and their parameters;
// rows at and past `n` read as zero and are not touched in memory.
struct TileSrc {
    const uint8_t *k, *v, *kp, *vp;  // the head's row 0
    int n;
};
__device__ __forceinline__ void issue_tile(const TileSrc& s, int tile, uint32_t stage, int lane) {
    const int row0 = tile * kTilePos;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int idx = lane + 32 * i, row = idx >> 2, c = idx & 3;
        const int bytes = row0 + row < s.n ? 16 : 0;
        const size_t off = bytes ? (size_t)(row0 + row) * kRowBytes + c * 16 : 0;
        cp_async16_zfill(stage + idx * 16, s.k + off, bytes);
        // V: the four rows of a lane in one 128-byte line position each, so
        // that the 8-byte reads below touch every bank once
        const int line = (row & 3) * 2 + (c >> 1), slot = 2 * (row >> 2) + (c & 1);
        cp_async16_zfill(stage + kStageV + line * 128 + slot * 16, s.v + off, bytes);
    }
    // one row's 8 bytes a lane (a head's parameters start on 8 bytes only when
    // max_pos is odd): lanes 0-15 K, 16-31 V
    const int row = row0 + (lane & 15), bytes = row < s.n ? 8 : 0;
    cp_async8_zfill(stage + kStagePar + lane * 8, (lane < 16 ? s.kp : s.vp) + (bytes ? (size_t)row * 8 : 0), bytes);
}

template <int G>
__global__ void __launch_bounds__(kAttnWarps * 32, 1) attn_kv4_kernel(const __grid_constant__ Kv4Params p) {
    extern __shared__ __align__(128) uint8_t ring[];
    __shared__ float qs[G][kHeadDim];               // log2(e) / sqrt(128) times the rotated queries
    __shared__ float knew[kHeadDim], vnew[kHeadDim];  // the new row as cached
    __shared__ float wm[kAttnWarps + 1][G], wl[kAttnWarps + 1][G];
    __shared__ float merge_c[kMaxSplitUnits][G];
    __shared__ float merge_l[G];
    __shared__ int s_last;

    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int r = lane >> 2, t = lane & 3;
    const int g = blockIdx.x / p.S, split = blockIdx.x % p.S;
    const bool has_new = split == p.S - 1;
    const size_t base = (size_t)g * p.max_pos;
    const int tile_end = min((p.pos + kTilePos - 1) / kTilePos, (split + 1) * p.tiles_per_split);

    const TileSrc src{p.k4 + base * kRowBytes, p.v4 + base * kRowBytes, reinterpret_cast<const uint8_t*>(p.k_par + base * 2),
                      reinterpret_cast<const uint8_t*>(p.v_par + base * 2), p.pos};
    uint8_t* my_ring = ring + warp * kRingBytes;
    const uint32_t my_ring_s = smem_u32(my_ring);
    int next = split * p.tiles_per_split + warp;  // next tile to copy
#pragma unroll
    for (int s = 0; s < kStages - 1; ++s) {
        if (next < tile_end) issue_tile(src, next, my_ring_s + s * kStageBytes, lane);
        cp_async_commit();
        next += kAttnWarps;
    }

    // queries: one warp per head; the new row: the last warp of the last split
    if (warp < G) {
        float q[4];
        norm_rope<float>(p.qkv + (size_t)(g * G + warp) * kHeadDim, p.q_norm, p.rope, p.eps, lane, q);
        const float c = 1.4426950408889634f / sqrtf((float)kHeadDim);
#pragma unroll
        for (int j = 0; j < 4; ++j) qs[warp][4 * lane + j] = q[j] * c;
    }
    if (has_new && warp == kAttnWarps - 1) {
        // the new key in fp64 up to its rounding to bf16: its 4-bit codes are
        // a step function of it, and must not depend on the order of a sum
        double kd[4];
        norm_rope<double>(p.qkv + (size_t)(p.n_q + g) * kHeadDim, p.k_norm, p.rope, p.eps, lane, kd);
        const float* vs = p.qkv + (size_t)(p.n_q + p.n_kv + g) * kHeadDim + 4 * lane;
        float kx[4], vx[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            kx[j] = round_bf16((float)kd[j]);
            vx[j] = round_bf16(vs[j]);
        }
        uint32_t kp, vp;
        const uint32_t kc = quant_row(kx, &kp), vc = quant_row(vx, &vp);
        const size_t at = base + p.pos;
        store_row(kc, kp, p.k4 + at * kRowBytes, p.k_par + at * 2, lane);
        store_row(vc, vp, p.v4 + at * kRowBytes, p.v_par + at * 2, lane);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float k = fmaf(bf16lo(kp), (float)((kc >> (4 * j)) & 15u), bf16hi(kp));
            const float v = fmaf(bf16lo(vp), (float)((vc >> (4 * j)) & 15u), bf16hi(vp));
            knew[4 * lane + j] = k;
            vnew[4 * lane + j] = v;
            if (p.kv_row) {
                p.kv_row[(size_t)g * kHeadDim + 4 * lane + j] = k;
                p.kv_row[(size_t)(p.n_kv + g) * kHeadDim + 4 * lane + j] = v;
            }
        }
    }
    __syncthreads();
    if (has_new && warp < G) {  // the new position: weight 1 at its own score
        float s = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) s = fmaf(qs[warp][4 * lane + j], knew[4 * lane + j], s);
        s = warp_sum(s);
        if (lane == 0) {
            wm[kAttnWarps][warp] = s;
            wl[kAttnWarps][warp] = 1.f;
        }
    }

    // query operand: word w of a K row's 16-byte piece t holds channels
    // 64 (w % 2) + 8 (2 t + w / 2) + 0..7; nibbles (0, 4), (1, 5) are the first
    // product's columns, (2, 6), (3, 7) the second's
    uint32_t qa[4][2][4];
    float fq = 0.f, qsum[2] = {0.f, 0.f};
    {
        float amax = 0.f;
        if (r < G) {
#pragma unroll
            for (int w = 0; w < 4; ++w)
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float q = qs[r][64 * (w & 1) + 8 * (2 * t + (w >> 1)) + i];
                    amax = fmaxf(amax, fabsf(q));
                    qsum[w & 1] += q;
                }
        }
#pragma unroll
        for (int o = 1; o <= 2; o <<= 1) {
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
            qsum[0] += __shfl_xor_sync(0xffffffffu, qsum[0], o);
            qsum[1] += __shfl_xor_sync(0xffffffffu, qsum[1], o);
        }
        const int e = expo(amax);
        const float f = to_2p15(e);
        fq = pow2_field(min(10 + e, 254));  // 2^24 / f
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            float q[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                q[i] = r < G ? qs[r][64 * (w & 1) + 8 * (2 * t + (w >> 1)) + i] * f : 0.f;
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                split_h2(q[2 * s], q[2 * s + 4], &qa[w][s][0], &qa[w][s][1]);
                split_h2(q[2 * s + 1] * 0.0625f, q[2 * s + 5] * 0.0625f, &qa[w][s][2], &qa[w][s][3]);
            }
        }
    }

    float M = -INFINITY, l = 0.f, wmax[2] = {0.f, 0.f}, fv[2] = {to_2p15(14), to_2p15(14)}, omin[2] = {0.f, 0.f};
    float o[2][8][4];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int c = 0; c < 4; ++c) o[h][i][c] = 0.f;

    int stage = 0;
    const int krow = 4 * (r >> 1) + (r & 1);
    const int voff = (r >> 2) * 128 + (2 * t + ((r >> 1) & 1)) * 16 + (r & 1) * 8;
    for (int tile = split * p.tiles_per_split + warp; tile < tile_end; tile += kAttnWarps) {
        cp_async_wait<kStages - 2>();
        __syncwarp();
        {
            int fill = stage + kStages - 1;
            if (fill >= kStages) fill -= kStages;
            if (next < tile_end) issue_tile(src, next, my_ring_s + fill * kStageBytes, lane);
            cp_async_commit();
            next += kAttnWarps;
        }
        const uint8_t* st = my_ring + stage * kStageBytes;
        if (++stage == kStages) stage = 0;

        // ---- scores of positions 4t .. 4t + 3 for head r
        float sc[4];
        const uint4 kpa = *reinterpret_cast<const uint4*>(st + kStagePar + t * 32);
        const uint4 kpb = *reinterpret_cast<const uint4*>(st + kStagePar + t * 32 + 16);
        const uint32_t kpar[4][2] = {{kpa.x, kpa.y}, {kpa.z, kpa.w}, {kpb.x, kpb.y}, {kpb.z, kpb.w}};
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            const uint4 w4 = *reinterpret_cast<const uint4*>(st + (krow + 2 * b) * kRowBytes + t * 16);
            const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
            float c[2][4] = {};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                mma16816(c[i & 1], qa[i][0], w[i] & 0x000f000fu, w[i] & 0x00f000f0u);
                mma16816(c[i & 1], qa[i][1], (w[i] >> 8) & 0x000f000fu, (w[i] >> 8) & 0x00f000f0u);
            }
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const uint32_t* kp = kpar[2 * b + j];
                const float x = fmaf(c[1][j] + c[1][2 + j], bf16lo(kp[1]), (c[0][j] + c[0][2 + j]) * bf16lo(kp[0]));
                sc[2 * b + j] = fmaf(x, fq, fmaf(bf16hi(kp[0]), qsum[0], bf16hi(kp[1]) * qsum[1]));
            }
        }
        if (tile * kTilePos + kTilePos > p.pos) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (tile * kTilePos + 4 * t + k >= p.pos) sc[k] = -INFINITY;
        }

        // ---- softmax weights, and the same times each position's V scale
        float mx = fmaxf(fmaxf(sc[0], sc[1]), fmaxf(sc[2], sc[3]));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        const float m_new = fmaxf(M, mx);
        const uint4 vpa = *reinterpret_cast<const uint4*>(st + kStagePar + 128 + t * 32);
        const uint4 vpb = *reinterpret_cast<const uint4*>(st + kStagePar + 128 + t * 32 + 16);
        const uint32_t vpar[4][2] = {{vpa.x, vpa.y}, {vpa.z, vpa.w}, {vpb.x, vpb.y}, {vpb.z, vpb.w}};
        float pw[4], ws[2][4], wx[2] = {0.f, 0.f}, lt = 0.f, ot[2] = {0.f, 0.f};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            pw[k] = ex2(sc[k] - m_new);
            lt += pw[k];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                ws[h][k] = pw[k] * bf16lo(vpar[k][h]);
                ot[h] = fmaf(pw[k], bf16hi(vpar[k][h]), ot[h]);
                wx[h] = fmaxf(wx[h], fabsf(ws[h][k]));
            }
        }
        wx[0] = fmaxf(wx[0], __shfl_xor_sync(0xffffffffu, wx[0], 1));
        wx[1] = fmaxf(wx[1], __shfl_xor_sync(0xffffffffu, wx[1], 1));
        wx[0] = fmaxf(wx[0], __shfl_xor_sync(0xffffffffu, wx[0], 2));
        wx[1] = fmaxf(wx[1], __shfl_xor_sync(0xffffffffu, wx[1], 2));
        const bool grew = m_new > M || expo(wx[0]) > expo(wmax[0]) || expo(wx[1]) > expo(wmax[1]);
        if (__any_sync(0xffffffffu, grew)) {
            const float corr = m_new > M ? ex2(M - m_new) : 1.f;
            l *= corr;
            M = m_new;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int e_old = expo(wmax[h]);
                wmax[h] = fmaxf(wmax[h] * corr, wx[h]);
                const int e_new = expo(wmax[h]);
                fv[h] = to_2p15(e_new);
                omin[h] *= corr;
                // 2^(e_old - e_new), past the smallest normal power: nothing is left
                const int d = 127 + e_old - e_new;
                const float k = corr * pow2_field(max(0, min(d, 254)));
#pragma unroll
                for (int i = 0; i < 8; ++i)
#pragma unroll
                    for (int c = 0; c < 4; ++c) o[h][i][c] *= k;
            }
        }
        l += lt;

        // ---- output: V rows 4t .. 4t + 3, channels 64 h + 8 r + i
        uint2 vw[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) vw[i] = *reinterpret_cast<const uint2*>(st + kStageV + voff + i * 256);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            omin[h] += ot[h];
            uint32_t a[4];
            split_h2(ws[h][0] * fv[h], ws[h][1] * fv[h], &a[0], &a[1]);
            split_h2(ws[h][2] * fv[h], ws[h][3] * fv[h], &a[2], &a[3]);
            const uint32_t w0 = h ? vw[0].y : vw[0].x, w1 = h ? vw[1].y : vw[1].x;
            const uint32_t w2 = h ? vw[2].y : vw[2].x, w3 = h ? vw[3].y : vw[3].x;
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const uint32_t sel = half ? 0x7632u : 0x5410u;
                const uint32_t x = __byte_perm(w0, w1, sel), y = __byte_perm(w2, w3, sel);
                mma16816(o[h][4 * half + 0], a, x & 0x000f000fu, y & 0x000f000fu);
                mma16816(o[h][4 * half + 1], a, x & 0x00f000f0u, y & 0x00f000f0u);
                mma16816(o[h][4 * half + 2], a, (x >> 8) & 0x000f000fu, (y >> 8) & 0x000f000fu);
                mma16816(o[h][4 * half + 3], a, (x >> 8) & 0x00f000f0u, (y >> 8) & 0x00f000f0u);
            }
        }
    }

    // ---- this warp's partial: maximum, sum, output (its ring is free now)
    cp_async_wait<0>();
    __syncwarp();
#pragma unroll
    for (int d = 1; d <= 2; d <<= 1) {
        l += __shfl_xor_sync(0xffffffffu, l, d);
        omin[0] += __shfl_xor_sync(0xffffffffu, omin[0], d);
        omin[1] += __shfl_xor_sync(0xffffffffu, omin[1], d);
    }
    if (r < G) {
        if (t == 0) {
            wm[warp][r] = M;
            wl[warp][r] = l;
        }
        float* po = reinterpret_cast<float*>(my_ring) + r * kHeadDim;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float back = pow2_field(expo(wmax[h]));  // 2^e, and 2^24 2^-14 = 2^10 below
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float k = i & 1 ? 64.f : 1024.f;
                po[64 * h + 8 * (2 * t) + i] = fmaf((o[h][i][0] + o[h][i][2]) * k, back, omin[h]);
                po[64 * h + 8 * (2 * t + 1) + i] = fmaf((o[h][i][1] + o[h][i][3]) * k, back, omin[h]);
            }
        }
    }
    __syncthreads();

    // ---- merge the warps and the new row.  A partial with sum 0 is empty; NaN
    // sums pass through.
    const int parts = has_new ? kAttnWarps + 1 : kAttnWarps;
    const size_t unit = (size_t)g * p.S + split;
    for (int idx = threadIdx.x; idx < G * kHeadDim; idx += kAttnWarps * 32) {
        const int j = idx / kHeadDim, d = idx % kHeadDim;
        float mx = -INFINITY;
        for (int w = 0; w < parts; ++w) mx = fmaxf(mx, wm[w][j]);
        float L = 0.f, O = 0.f;
        for (int w = 0; w < parts; ++w) {
            if (wl[w][j] == 0.f) continue;
            const float c = ex2(wm[w][j] - mx);
            L += wl[w][j] * c;
            O += (w < kAttnWarps ? reinterpret_cast<const float*>(ring + w * kRingBytes)[idx] : vnew[d]) * c;
        }
        if (p.S == 1) {
            p.out[(size_t)g * G * kHeadDim + idx] = O / L;
        } else {
            p.part_o[unit * G * kHeadDim + idx] = O;
            if (d == 0) p.part_ml[unit * G + j] = make_float2(mx, L);
        }
    }
    if (p.S == 1) return;

    // ---- the last split of this kv head to finish merges all splits, in order
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) s_last = atomicAdd(&p.tickets[g], 1u) == (unsigned)(p.S - 1);
    __syncthreads();
    if (!s_last) return;
    __threadfence();
    const float2* ml = p.part_ml + (size_t)g * p.S * G;
    if (warp < G) {
        float mx = -INFINITY;
        for (int s = lane; s < p.S; s += 32) mx = fmaxf(mx, __ldcg(&ml[s * G + warp]).x);
        mx = warp_max(mx);
        float L = 0.f;
        for (int s = lane; s < p.S; s += 32) {
            const float2 v = __ldcg(&ml[s * G + warp]);
            const float c = ex2(v.x - mx);
            merge_c[s][warp] = c;
            L += v.y * c;
        }
        L = warp_sum(L);
        if (lane == 0) merge_l[warp] = L;
    }
    __syncthreads();
    const float* po = p.part_o + (size_t)g * p.S * G * kHeadDim;
    for (int idx = threadIdx.x; idx < G * kHeadDim; idx += kAttnWarps * 32) {
        const int j = idx / kHeadDim;
        float O = 0.f;
#pragma unroll 8
        for (int s = 0; s < p.S; ++s) O = fmaf(__ldcg(po + (size_t)s * G * kHeadDim + idx), merge_c[s][j], O);
        p.out[(size_t)g * G * kHeadDim + idx] = O / merge_l[j];
    }
    if (threadIdx.x == 0) p.tickets[g] = 0u;
}

template <int G>
cudaError_t launch_attn_kv4(const Kv4Params& p, cudaStream_t s) {
    static std::atomic<unsigned long long> ready{0};  // devices whose shared-memory limit is raised
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const unsigned long long bit = 1ull << (dev & 63);
    if (!(ready.load(std::memory_order_relaxed) & bit)) {
        e = cudaFuncSetAttribute(attn_kv4_kernel<G>, cudaFuncAttributeMaxDynamicSharedMemorySize, kAttnSmem);
        if (e != cudaSuccess) return e;
        ready.fetch_or(bit, std::memory_order_relaxed);
    }
    attn_kv4_kernel<G><<<p.n_kv * p.S, kAttnWarps * 32, kAttnSmem, s>>>(p);
    return cudaGetLastError();
}

bool misaligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0; }

int report_kv4(cudaError_t e, const char* what) {
    std::fprintf(stderr, "tts: %s failed: %s\n", what, cudaGetErrorString(e));
    return TTS_ERR_CUDA;
}

int max_splits(int n_kv) { return n_kv >= kMaxSplitUnits ? 1 : kMaxSplitUnits / n_kv; }

// [tickets][maximum and sum: 2 words per split and query head][outputs: 128
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

int rows_ok(const void* k, const void* v, const void* k4, const void* v4, const void* kp, const void* vp, int n_kv,
            int p0, int p1, int stride, int max_pos) {
    if (!k || !v || !k4 || !v4 || !kp || !vp || n_kv < 1 || n_kv > kKv4MaxKvHeads) return TTS_ERR_ARG;
    if (max_pos < 1 || max_pos > kKv4MaxPos || p0 < 0 || p1 < p0) return TTS_ERR_ARG;
    if (misaligned(k, 16) || misaligned(v, 16) || misaligned(k4, 16) || misaligned(v4, 16) || misaligned(kp, 16) ||
        misaligned(vp, 16))
        return TTS_ERR_ARG;
    if (p1 > max_pos) return TTS_ERR_FULL;
    if (p1 > stride) return TTS_ERR_ARG;
    return TTS_OK;
}

}  // namespace
}  // namespace tts

extern "C" int tts_quantize_kv4(const void* k, const void* v, int n_kv, int p0, int p1, int src_stride, void* k4,
                                void* v4, void* k_par, void* v_par, int max_pos, void* stream) {
    using namespace tts;
    const int rc = rows_ok(k, v, k4, v4, k_par, v_par, n_kv, p0, p1, src_stride, max_pos);
    if (rc != TTS_OK || p0 == p1) return rc;
    const dim3 grid((p1 - p0 + 7) / 8, 2 * n_kv);
    quantize_kv4_kernel<<<grid, 256, 0, static_cast<cudaStream_t>(stream)>>>(
        static_cast<const uint16_t*>(k), static_cast<const uint16_t*>(v), n_kv, p0, p1 - p0, src_stride,
        static_cast<uint8_t*>(k4), static_cast<uint8_t*>(v4), static_cast<uint32_t*>(k_par),
        static_cast<uint32_t*>(v_par), max_pos);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? TTS_OK : report_kv4(e, "tts_quantize_kv4");
}

extern "C" int tts_dequantize_kv4(const void* k4, const void* v4, const void* k_par, const void* v_par, int n_kv,
                                  int p0, int p1, int max_pos, void* k, void* v, int dst_stride, void* stream) {
    using namespace tts;
    const int rc = rows_ok(k, v, k4, v4, k_par, v_par, n_kv, p0, p1, dst_stride, max_pos);
    if (rc != TTS_OK || p0 == p1) return rc;
    const dim3 grid((p1 - p0 + 7) / 8, 2 * n_kv);
    dequantize_kv4_kernel<<<grid, 256, 0, static_cast<cudaStream_t>(stream)>>>(
        static_cast<const uint8_t*>(k4), static_cast<const uint8_t*>(v4), static_cast<const uint32_t*>(k_par),
        static_cast<const uint32_t*>(v_par), n_kv, p0, p1 - p0, max_pos, static_cast<uint16_t*>(k),
        static_cast<uint16_t*>(v), dst_stride);
    const cudaError_t e = cudaGetLastError();
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
    for (int i = 0; i < kHeadDim / 2; ++i) {
        const double ang = (double)pos * std::pow((double)rope_theta, -2.0 * i / (double)kHeadDim);
        const double c = std::cos(ang), sn = std::sin(ang);
        p.rope.cs[i] = make_float2((float)c, (float)sn);
        p.rope.rest[i] = make_float2((float)(c - (double)(float)c), (float)(sn - (double)(float)sn));
    }
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return TTS_ERR_CUDA;
    // splits: at most one block per SM over all kv heads, at least a tile for
    // every warp of a block, none empty
    const int tiles = (pos + kTilePos - 1) / kTilePos;
    int S = (tiles + kAttnWarps - 1) / kAttnWarps;
    S = std::max(1, std::min(S, std::min(max_splits(n_kv), sms / n_kv)));
    p.tiles_per_split = std::max(1, (tiles + S - 1) / S);
    p.S = std::max(1, (tiles + p.tiles_per_split - 1) / p.tiles_per_split);
    char* ws = static_cast<char*>(workspace);
    p.tickets = reinterpret_cast<unsigned*>(ws);
    p.part_ml = reinterpret_cast<float2*>(ws + kTicketBytes);
    p.part_o = reinterpret_cast<float*>(ws + kTicketBytes + sizeof(float2) * (size_t)n_q * max_splits(n_kv));
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    switch (n_q / n_kv) {
        case 1: e = launch_attn_kv4<1>(p, st); break;
        case 2: e = launch_attn_kv4<2>(p, st); break;
        case 4: e = launch_attn_kv4<4>(p, st); break;
        default: e = launch_attn_kv4<8>(p, st); break;
    }
    return e == cudaSuccess ? TTS_OK : report_kv4(e, "tts_attention_decode_kv4");
}
