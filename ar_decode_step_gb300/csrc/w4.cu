// 4-bit weights with group scales: quantisation of a bf16 matrix and the
// matrix-vector product of a decode step (sm_103a).
//
// Format: W4 uint8 [N][K/2], low nibble = even k, u in 0..15; s bf16
// [N][K/128]; weight = s * (u - 8).
#include <algorithm>
#include <cmath>
#include <cstdio>
#include <mutex>
#include <type_traits>

#include <cooperative_groups.h>

#include "fourbit.cuh"
#include "tts_decode.h"

namespace tts {
namespace {

constexpr int kW4Group = 128;
constexpr int kW4MaxM = 8;
constexpr int kW4MaxK = 12288;

struct W4Params {
    const float* x;
    const uint8_t* W4;
    const __nv_bfloat16* s;
    const float* resid;
    const __nv_bfloat16* gamma;
    float* y;
    int M, N, K, epi;
    float eps;
};

// One warp per group of 128 weights: lane l holds k = 4l .. 4l + 3.
// s = bf16(amax / 7): both the division and the quotients w / s are IEEE
// fp32, so that every side that follows the definition gets the same codes
// (w and s have 8 significant bits: the fp32 quotient never crosses a
// rounding border that the exact one does not).
__global__ void __launch_bounds__(256) quantize_w4_kernel(const __nv_bfloat16* __restrict__ W, size_t groups,
                                                          uint8_t* __restrict__ W4, __nv_bfloat16* __restrict__ s) {
    const int lane = threadIdx.x & 31;
    const size_t g = (size_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (g >= groups) return;
    const uint16_t* src = reinterpret_cast<const uint16_t*>(W) + g * kW4Group + 4 * lane;
    const uint2 w = *reinterpret_cast<const uint2*>(src);
    const float v[4] = {bf16lo(w.x), bf16hi(w.x), bf16lo(w.y), bf16hi(w.y)};
    const float amax = warp_max(fmaxf(fmaxf(fabsf(v[0]), fabsf(v[1])), fmaxf(fabsf(v[2]), fabsf(v[3]))));
    const __nv_bfloat16 sb = __float2bfloat16_rn(__fdiv_rn(amax, 7.f));
    const float sc = __bfloat162float(sb);
    uint32_t code = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float q = sc > 0.f ? fminf(fmaxf(rintf(__fdiv_rn(v[j], sc)), -8.f), 7.f) : 0.f;
        code |= (uint32_t)((int)q + 8) << (4 * j);
    }
    *reinterpret_cast<uint16_t*>(W4 + g * (kW4Group / 2) + 2 * lane) = (uint16_t)code;
    if (lane == 0) s[g] = sb;
}

// ---- the product -----------------------------------------------------------------
// y[m][n] = sum_k a[m][k] s[n][k/128] (u[n][k] - 8).  Its time is the reading of
// the weights once (at most 16 flops a byte), so everything else has to stay
// below that: a weight may cost about 2.7 of an SM's lane instructions.
//
// Codes are the A operand of m16n8k16 products (fp16, fp32 sums), centred: u - 8
// and, from a whole byte, (u - 8) + 16 (u' - 8), exact in fp16, one logical and one
// fp16 instruction per two of them; a (u - 8) + a' (u' - 8) = (a - a'/16)(u - 8) +
// (a'/16)((u - 8) + 16 (u' - 8)) moves the rest to the activations.  These are
// the B operand: fp32, scaled per 128 group by a power of two to below 2^15 and
// split into two fp16 parts (22 bits, and 2^-39 of the group's largest).  Up to
// four vectors take columns 2m and 2m + 1 of one product, eight a product for each
// part.  Group sums leave the tensor core once a group and are scaled and added
// in fp32.
//
// About one block an SM.  A block takes tiles of 16 rows (epi 2: a gate and an up
// tile) of all of K, or of a share of K where its activations or its tiles would
// not fit the SM (a cluster of blocks then adds up through distributed shared
// memory).  All its rows are copied at once by the bulk-copy engine, one copy a
// row, to rows 64 bytes apart modulo 128, so that the 16-byte reads of eight
// lanes (two rows, four pieces) touch every bank once; a barrier a tile says
// when it is there, and nothing is ever overwritten.  A warp has one slice of
// the groups for all tiles, so it prepares its slice of the activations once and
// for itself, while the first rows are on their way; the warps' sums are added
// at the end.
// (Measured first, gate/up at one vector: small blocks, four an SM, 11.7 us, most
// of it preparing the same activations four times; 16-byte asynchronous copies by
// the lanes, 10.9 us, of which 3 us to issue them: 40 cache lines an item.)
constexpr int kMaxTiles = 8;  // tiles (epi 2: pairs) a block, at most

struct W4Launch {
    int warps, tiles, share, log_split;  // tiles a block, groups of K a block at most, log2 of the blocks that share K
    int grid;
    unsigned long long magic;  // ceil(2^32 / warps): n / warps = n magic >> 32 for the small n here
    size_t smem;
};

__device__ __forceinline__ void mma16816_f16(float c[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                             uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// d = A B, without clearing d first
__device__ __forceinline__ void mma16816_f16_first(float c[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                                   uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

// Shared memory of a block: [rows: tiles x parts x 16][activations: share x 4 words
// x columns x 4 pieces x 16 bytes][per group and vector: 1 over its power of
// two][scales: tiles x parts x share x 16 bf16][sums: outputs x parts x
// warps][sums of squares: MV x warps][totals of the block: outputs x parts, MV].
__host__ __device__ constexpr int columns_of(int mv) { return 2 * mv; }
__host__ __device__ constexpr int act_group_bytes(int mv) { return 4 * columns_of(mv) * 64; }
// Kernels of four vectors with a gate and an up tile come in two forms: a warp's sums in
// a place of their own, or (in_act) where its first group's activations were, which
// are in registers by then.  The second is 5 to 17 % slower at equal plans (gate/up
// 6144 x 2560 8.2 us against 7.7, 4096 x 2048 5.9 and 5.5, 2560 x 9728 20.7 and 17.4)
// and saves 41 KB a block of four tiles: it is taken where that saves a round of
// blocks (9728 x 2560 10.2 against 14.7, 16384 x 2560 19.0 and 22.1).  Elsewhere a
// round is not to be had.
__host__ __device__ constexpr bool has_in_act(int mv, int parts) { return mv == 4 && parts == 2; }
// (20 at eight vectors, in 96 registers, took 8.6 us instead of 8.2 on 8208 x 2560.)
__host__ __device__ constexpr int max_warps(int mv) { return mv == 8 ? 16 : 20; }
__host__ __device__ inline int row_pitch(int share) { return share * 64 + (share & 1 ? 0 : 64); }
struct W4Smem {
    uint32_t act, par, scales, sums, sq, tot, total;
};
__host__ __device__ inline W4Smem smem_of(int mv, int parts, bool in_act, int tiles, int share, int warps) {
    W4Smem o;
    const uint32_t outs = tiles * 16 * mv * parts;
    o.act = tiles * parts * 16 * row_pitch(share);
    o.par = o.act + share * act_group_bytes(mv);
    o.scales = (o.par + share * mv * 4 + 15) & ~15u;
    o.sums = o.scales + tiles * parts * share * 32;
    o.sq = o.sums + (in_act ? 0 : outs * warps * 4);
    o.tot = o.sq + mv * warps * 4;
    o.total = o.tot + (outs + mv) * 4;
    return o;
}

template <int MV, int PARTS, bool IN_ACT>  // vectors (1, 2, 4, 8), tiles an output tile takes, the sums' place
__global__ void __launch_bounds__(max_warps(MV) * 32, 1) gemv_w4_kernel(const W4Params p, const W4Launch c) {
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ __align__(8) uint64_t bars[kMaxTiles * PARTS];
    __shared__ int late;  // a tile did not arrive: the outputs are NaN
    constexpr int kVecs = MV == 8 ? 2 : 1;  // vectors a lane adds up
    const int lane = threadIdx.x & 31, warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), W = c.warps;
    const int r = lane >> 2, t = lane & 3;
    const int groups = p.K / kW4Group, rank = blockIdx.z, split = 1 << c.log_split;
    const int k0 = groups * rank >> c.log_split, kg = (groups * (rank + 1) >> c.log_split) - k0;  // this block's groups of K
    // this warp's of those; where they do not come out even, the last warps have one
    // more: they copy no rows, and neighbours are on different schedulers (8208 x 2560 at
    // eight vectors, 20 groups for 16 warps: 8.2 us; 10.1 with every fourth warp, all of
    // one scheduler, having two)
    const int each = (int)(kg * c.magic >> 32), even = W - (kg - each * W);
    auto first_of = [&](int w) { return each * w + max(w - even, 0); };
    const int g0 = first_of(warp), g1 = first_of(warp + 1);
    const int ntiles = (p.N + 15) / 16;
    const int tile0 = blockIdx.x, step = gridDim.x;
    // this block's tiles: tile0, tile0 + step, ...
    const int nt = c.tiles - ((long long)tile0 + (long long)(c.tiles - 1) * step >= ntiles);
    const int pitch = row_pitch(c.share);
    const W4Smem o = smem_of(MV, PARTS, IN_ACT, c.tiles, c.share, W);

    // ---- activations of the slice's first group, then the copies
    float4 xs[MV];
    uint2 gb = {};
    auto load_x = [&](int g) {
        const size_t k = (size_t)(k0 + g) * kW4Group + 4 * lane;
#pragma unroll
        for (int m = 0; m < MV; ++m)
            xs[m] = m < p.M ? *reinterpret_cast<const float4*>(p.x + (size_t)m * p.K + k) : make_float4(0.f, 0.f, 0.f, 0.f);
        if (p.gamma) gb = *reinterpret_cast<const uint2*>(p.gamma + k);
    };
    if (threadIdx.x == 0) {
        for (int q = 0; q < nt * PARTS; ++q) mbar_init(&bars[q], 1);
        late = 0;
        fence_mbar_init();
    }
    __syncthreads();
    if (split > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
    pdl_trigger();
    pdl_wait();
    if (g0 < g1) load_x(g0);
    // row i of the block's tile q; past the end the last row, whose result is not
    // stored
    auto row_of = [&](int q, int i) {
        return min((tile0 + q / PARTS * step) * 16 + i, p.N - 1) + (q % PARTS) * p.N;
    };
    // Scales, bf16 [tile x parts][16][share].  With all of K a tile's are one run of
    // 32 bytes a group and come with its rows, but for a last tile of fewer rows and
    // a run that does not start on 16 bytes.  Otherwise a row a warp at a time, eight
    // rows in flight, the first before the copies, which would hold them up for 2 us.
    __nv_bfloat16* scl = reinterpret_cast<__nv_bfloat16*>(smem + o.scales);
    auto run_of = [&](int q) { return p.s + (size_t)row_of(q, 0) * groups; };
    auto in_run = [&](int q) {
        return split == 1 && (tile0 + q / PARTS * step) * 16 + 16 <= p.N && (reinterpret_cast<uintptr_t>(run_of(q)) & 15) == 0;
    };
    constexpr int kAhead = 8;
    const int rows = nt * PARTS * 16;
    __nv_bfloat16 sv[kAhead];
    auto load_scales = [&](int i0, int gl) {
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            const int i = min(i0 + j * W, rows - 1);  // past the end the last row again
            if (gl < kg) sv[j] = p.s[(size_t)row_of(i >> 4, i & 15) * groups + k0 + gl];
        }
    };
    auto keep_scales = [&](int i0, int gl) {
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            const int i = i0 + j * W;
            if (i < rows && gl < kg) scl[i * c.share + gl] = sv[j];
        }
    };
    if (split > 1) load_scales(warp, lane);
    // Rows spread over the warps, but at four and eight vectors a tile's to one warp:
    // each copy holds its warp up for about 60 ns, and there the others' preparation is
    // what the products wait for (gate/up at one vector 9.4 us spread, 9.8 otherwise;
    // 8208 x 2560 at eight 8.5 and 8.15).
    constexpr bool kSpread = MV <= 2;
    const uint64_t once = l2_evict_first_policy();
    for (int q = warp; q < nt * PARTS; q += W) {
        const bool run = in_run(q);
        if (lane == 0) mbar_arrive_expect_tx(&bars[q], 16 * kg * 64 + (run ? 32 * groups : 0));
        if (lane == 16 && run) bulk_g2s(scl + (size_t)q * 16 * groups, run_of(q), 32 * groups, &bars[q], once);
    }
    if (kSpread || lane < 16)
        for (int i = kSpread ? warp + W * lane : warp * 16 + lane; i < rows; i += W * (kSpread ? 32 : 16))
            bulk_g2s(smem + (size_t)i * pitch, p.W4 + (size_t)row_of(i >> 4, i & 15) * (p.K / 2) + k0 * 64, kg * 64,
                     &bars[i >> 4], once);
    __syncwarp();
    if (split > 1) {
        keep_scales(warp, lane);
        for (int gl = lane; gl < kg; gl += 32)
            for (int i0 = gl == lane ? warp + kAhead * W : warp; i0 < rows; i0 += kAhead * W) {
                load_scales(i0, gl);
                keep_scales(i0, gl);
            }
    } else {
        for (int q = 0; q < nt * PARTS; ++q)
            if (!in_run(q))
                for (int i = warp; i < 16; i += W)
                    for (int g = lane; g < kg; g += 32)
                        scl[(q * 16 + i) * c.share + g] = p.s[(size_t)row_of(q, i) * groups + g];
    }

    // a thread adds up output i = its number, + threads, ... at the end: what it
    // adds the first of them to
    const int outs = nt * 16 * MV;
    auto place = [&](int i, size_t* at) {  // output i: (tile, row, vector)
        const int n = (tile0 + i / (16 * MV) * step) * 16 + (i / MV) % 16, m = i % MV;
        *at = (size_t)m * p.N + n;
        return i < outs && n < p.N && m < p.M;
    };
    float resid = 0.f;
    if (p.resid && split == 1) {
        size_t at;
        if (place(threadIdx.x, &at)) resid = p.resid[at];
    }

    // ---- this warp's slice of the activations
    float* act_par = reinterpret_cast<float*>(smem + o.par);
    float* sq = reinterpret_cast<float*>(smem + o.sq);  // [W][MV]
    float ss[MV];
#pragma unroll
    for (int m = 0; m < MV; ++m) ss[m] = 0.f;
    for (int g = g0; g < g1; ++g) {
        float a[MV][4];
#pragma unroll
        for (int m = 0; m < MV; ++m) {
            a[m][0] = xs[m].x;
            a[m][1] = xs[m].y;
            a[m][2] = xs[m].z;
            a[m][3] = xs[m].w;
            if (p.gamma) {
#pragma unroll
                for (int j = 0; j < 4; ++j) ss[m] = fmaf(a[m][j], a[m][j], ss[m]);
                a[m][0] *= bf16lo(gb.x);
                a[m][1] *= bf16hi(gb.x);
                a[m][2] *= bf16lo(gb.y);
                a[m][3] *= bf16hi(gb.y);
            }
        }
        if (g + 1 < g1) load_x(g + 1);
        uint8_t* dst = smem + o.act + (size_t)g * act_group_bytes(MV) + ((lane >> 1) & 3) * (columns_of(MV) * 64) +
                       (lane >> 3) * 16 + (lane & 1) * 8;
#pragma unroll
        for (int m = 0; m < MV; ++m) {
            const uint32_t amax = __reduce_max_sync(
                0xffffffffu,
                __float_as_uint(fmaxf(fmaxf(fabsf(a[m][0]), fabsf(a[m][1])), fmaxf(fabsf(a[m][2]), fabsf(a[m][3])))));
            // the group's power of two: largest to [2^14, 2^15)
            const int e = max((int)(amax >> 23), 15);
            const float f = __uint_as_float((uint32_t)(268 - e) << 23);
            if (lane == 0) act_par[g * MV + m] = __uint_as_float((uint32_t)(e - 14) << 23);  // 1 / f
            // channels 4 l .. 4 l + 3 are nibbles 4 (l % 2) + 0..3 of word (l / 2) % 4 of
            // piece l / 8: of the pairs (0, 4), (1, 5), (2, 6), (3, 7) an even lane
            // has the low halves, an odd lane the high ones
            uint32_t hi[2], lo[2];  // (pair 0, pair 1), (pair 2, pair 3)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                // (scaled first: a - a' / 16 of the largest numbers would overflow)
                const float v1 = a[m][2 * j + 1] * (0.0625f * f), v0 = fmaf(a[m][2 * j], f, -v1);
                const __half2 h = __floats2half2_rn(v0, v1);
                const float2 hf = __half22float2(h);
                const __half2 l = __floats2half2_rn(v0 - hf.x, v1 - hf.y);
                hi[j] = *reinterpret_cast<const uint32_t*>(&h);
                lo[j] = *reinterpret_cast<const uint32_t*>(&l);
            }
            const bool odd = lane & 1;
            const uint32_t gh = __shfl_xor_sync(0xffffffffu, odd ? hi[0] : hi[1], 1);
            const uint32_t gl = __shfl_xor_sync(0xffffffffu, odd ? lo[0] : lo[1], 1);
            const uint32_t eh = odd ? gh : hi[0], oh = odd ? hi[1] : gh;  // the even and the odd lane's halves
            const uint32_t el = odd ? gl : lo[0], ol = odd ? lo[1] : gl;
            uint8_t* d = dst + (MV == 8 ? m : 2 * m) * 64;
            *reinterpret_cast<uint2*>(d) = make_uint2(__byte_perm(eh, oh, 0x5410), __byte_perm(eh, oh, 0x7632));
            *reinterpret_cast<uint2*>(d + (MV == 8 ? 512 : 64)) = make_uint2(__byte_perm(el, ol, 0x5410), __byte_perm(el, ol, 0x7632));
        }
    }
    if (p.gamma) {
#pragma unroll
        for (int m = 0; m < MV; ++m) {
            ss[m] = warp_sum(ss[m]);
            if (lane == 0) sq[warp * MV + m] = ss[m];
        }
    }
    __syncthreads();  // the scales come from other warps

    // ---- the products: a group's activations in registers, all tiles past them
    static_assert(!IN_ACT || kMaxTiles / 2 * 16 * MV * PARTS * 4 <= act_group_bytes(MV), "a warp's sums fit a group");
    float* sums = IN_ACT ? reinterpret_cast<float*>(smem + o.act + g0 * act_group_bytes(MV))
                         : reinterpret_cast<float*>(smem + o.sums) + (size_t)warp * outs * PARTS;  // [tile x parts][row][vector]
    const bool column = MV == 8 || r < 2 * MV;
    for (int g = g0; g < g1; ++g) {
        uint4 b[kVecs][4];
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            const uint8_t* at = smem + o.act + (size_t)g * act_group_bytes(MV) + w * (columns_of(MV) * 64) + r * 64 + t * 16;
            b[0][w] = column ? *reinterpret_cast<const uint4*>(at) : make_uint4(0, 0, 0, 0);
            if (MV == 8) b[kVecs - 1][w] = *reinterpret_cast<const uint4*>(at + 512);
        }
        float ap[kVecs];
#pragma unroll
        for (int v = 0; v < kVecs; ++v) ap[v] = act_par[g * MV + min(kVecs * t + v, MV - 1)];
        if (IN_ACT && g == g0) __syncwarp();  // all lanes have read what the sums replace
        const uint8_t* row = smem + r * pitch + t * 16 + g * 64;
        const __nv_bfloat16* sc = scl + r * c.share + g;
        float* out = sums + r * MV + kVecs * t;
        // n tiles at a time: their loads, conversions and products are independent
        auto tiles = [&](int q, auto n_) {
            constexpr int n = decltype(n_)::value;
            if (g == g0) {
#pragma unroll
                for (int k = 0; k < n; ++k)
                    if (!mbar_arrived(&bars[q + k])) late = 1;
            }
            uint4 wa[n], wb[n];
            float sa[n], sb[n], d[n][2][4];
#pragma unroll
            for (int k = 0; k < n; ++k) {
                wa[k] = *reinterpret_cast<const uint4*>(row + k * 16 * pitch);
                wb[k] = *reinterpret_cast<const uint4*>(row + (k * 16 + 8) * pitch);
                sa[k] = __bfloat162float(sc[k * 16 * c.share]);
                sb[k] = __bfloat162float(sc[(k * 16 + 8) * c.share]);
            }
            row += n * 16 * pitch;
            sc += n * 16 * c.share;
#pragma unroll
            for (int w = 0; w < 4; ++w)
#pragma unroll
                for (int k = 0; k < n; ++k) {
                    const uint32_t ua = w == 0 ? wa[k].x : w == 1 ? wa[k].y : w == 2 ? wa[k].z : wa[k].w;
                    const uint32_t ub = w == 0 ? wb[k].x : w == 1 ? wb[k].y : w == 2 ? wb[k].z : wb[k].w;
#pragma unroll
                    for (int odd = 0; odd < 2; ++odd) {
                        const uint32_t x = nibble_bytes(ua, odd), y = nibble_bytes(ub, odd);
                        const uint32_t xl = low_code(x), yl = low_code(y), xb = both_codes(x), yb = both_codes(y);
#pragma unroll
                        for (int v = 0; v < kVecs; ++v) {
                            const uint32_t b0 = odd ? b[v][w].z : b[v][w].x, b1 = odd ? b[v][w].w : b[v][w].y;
                            if (w == 0 && v == 0)
                                mma16816_f16_first(d[k][odd], xl, yl, xb, yb, b0, b1);
                            else
                                mma16816_f16(d[k][odd], xl, yl, xb, yb, b0, b1);
                        }
                    }
                }
#pragma unroll
            for (int k = 0; k < n; ++k) {
                float y[2][kVecs];
#pragma unroll
                for (int v = 0; v < kVecs; ++v)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        float x;
                        if (MV == 8)
                            x = d[k][0][2 * h + v] + d[k][1][2 * h + v];
                        else
                            x = (d[k][0][2 * h] + d[k][1][2 * h]) + (d[k][0][2 * h + 1] + d[k][1][2 * h + 1]);
                        // the scales first: exact to 2^-149, while the sum of a (u - 8) of
                        // activations above 2^117 may be beyond fp32
                        y[h][v] = (h ? sb[k] : sa[k]) * ap[v] * x;
                    }
                if (MV == 8 || t < MV) {
#pragma unroll
                    for (int v = 0; v < kVecs; ++v)
#pragma unroll
                        for (int h = 0; h < 2; ++h) out[h * 8 * MV + v] = g == g0 ? y[h][v] : out[h * 8 * MV + v] + y[h][v];
                }
                out += 16 * MV;
            }
        };
        int q = 0;
        for (; q + 2 <= nt * PARTS; q += 2) tiles(q, std::integral_constant<int, 2>{});
        if (q < nt * PARTS) tiles(q, std::integral_constant<int, 1>{});
    }
    if (!IN_ACT && g0 == g1)  // no group: nothing of this warp's, but its copies
        for (int i = lane; i < outs * PARTS; i += 32) sums[i] = 0.f;
    for (int q = 0; q < nt * PARTS; ++q)
        if (g0 == g1 && !mbar_arrived(&bars[q])) late = 1;
    __syncthreads();
    if (late)  // a copy may still be on its way: once more, again with a limit
        for (int q = 0; q < nt * PARTS; ++q) mbar_wait(&bars[q], 0);

    // ---- the warps' sums in order, an output a thread
    const float* all = reinterpret_cast<const float*>(smem + o.sums);
    float* tot = reinterpret_cast<float*>(smem + o.tot);  // [MV] squares, [tile][part][row][vector]
    auto store = [&](size_t at, float v0, float v1, float squares, float add) {
        const float rms = p.gamma ? 1.f / sqrtf(squares / (float)p.K + p.eps) : 1.f;
        float y = v0 * rms + add;
        if (PARTS == 2) y = y / (1.f + expf(-y)) * (v1 * rms);
        p.y[at] = late ? NAN : y;
    };
    for (int i = threadIdx.x; i < outs; i += W * 32) {
        const int first = i + i / (16 * MV) * (16 * MV) * (PARTS - 1);  // part 0 of output i
        float v[PARTS] = {}, squares = 0.f;
#pragma unroll 4
        for (int w = 0; w < W; ++w) {
#pragma unroll
            for (int h = 0; h < PARTS; ++h)
                if (!IN_ACT) {
                    v[h] += all[(size_t)w * outs * PARTS + first + h * 16 * MV];
                } else {  // where warp w's first group was, if it had any
                    const int from = first_of(w), to = first_of(w + 1);
                    const float* theirs = reinterpret_cast<const float*>(smem + o.act + from * act_group_bytes(MV));
                    if (from < to) v[h] += theirs[first + h * 16 * MV];
                }
            if (p.gamma) squares += sq[w * MV + i % MV];
        }
        if (split == 1) {
            size_t at;
            if (place(i, &at)) store(at, v[0], v[PARTS - 1], squares, p.resid ? (i < W * 32 ? resid : p.resid[at]) : 0.f);
        } else {
            if (i < MV) tot[i] = squares;
#pragma unroll
            for (int h = 0; h < PARTS; ++h) tot[MV + first + h * 16 * MV] = late ? NAN : v[h];
        }
    }
    if (split == 1) return;

    // ---- the blocks' totals, outputs in turn by the blocks of the cluster
    asm volatile("barrier.cluster.wait.aligned;" ::: "memory");  // all blocks run
    const auto cluster = cooperative_groups::this_cluster();
    cluster.sync();
    for (int i = (int)threadIdx.x * split + rank; i < outs; i += W * 32 * split) {
        const int first = i + i / (16 * MV) * (16 * MV) * (PARTS - 1);
        float v[PARTS] = {}, squares = 0.f;
        for (int k = 0; k < split; ++k) {
            const float* theirs = cluster.map_shared_rank(tot, k);
            squares += theirs[i % MV];
#pragma unroll
            for (int h = 0; h < PARTS; ++h) v[h] += theirs[MV + first + h * 16 * MV];
        }
        size_t at;
        if (place(i, &at)) store(at, v[0], v[PARTS - 1], squares, p.resid ? p.resid[at] : 0.f);
    }
    cluster.sync();  // before a block's shared memory goes
}

constexpr size_t kBlockSmem = 227 * 1024 - 1024;  // the barriers' share left out

// Blocks, warps a block, tiles a block and the split of K for p at MV vectors;
// at_once[i]: clusters of 2^i blocks of this kernel that run at once.
W4Launch plan_gemv_w4(const W4Params& p, int mv, int parts, bool in_act, const int at_once[4]) {
    const int groups = p.K / kW4Group, ntiles = (p.N + 15) / 16, most_tiles = in_act ? kMaxTiles / 2 : kMaxTiles;
    auto made = [&](int log_split, int tiles, int grid) {
        const int share = (groups + (1 << log_split) - 1) >> log_split, warps = std::min(share, max_warps(mv));
        return W4Launch{warps, tiles, share, log_split, grid, ((1ull << 32) + warps - 1) / warps,
                        smem_of(mv, parts, in_act, tiles, share, warps).total};
    };
    // All tiles resident at once, a block an SM, K split so that the estimate is
    // least: a warp's turns (groups of K, between the most a warp has and the mean)
    // times its tiles and the preparation of its vectors, and 2.2 tiles for joining
    // a cluster.  2560 x 9728 at 1, 2, 4 vectors: K in four 7.7, 7.7, 7.9 us, the least
    // split that fits 8.0, 8.7, 9.2; 2560 x 4096: K whole 4.6, 4.9, 5.4 against 5.4, 5.4, 5.7
    // in two, at 8 vectors 7.8 against 7.1.  (Clusters of 3, 5 and 6 blocks were
    // slower than of 4 and 8 throughout.)
    int end = 1;  // of the splits whose clusters the device has room for
    while (end < 4 && (1 << end) <= groups && at_once[end] > 0) ++end;
    W4Launch best{};
    float least = 0.f;
    for (int ls = 0; ls < end; ++ls) {
        const int most = std::max(1, std::min(ntiles, at_once[ls])), tiles = (ntiles + most - 1) / most;
        if (tiles > most_tiles) continue;
        const W4Launch c = made(ls, tiles, most);
        if (c.smem > kBlockSmem) continue;
        const float turns = 0.5f * ((float)((c.share + c.warps - 1) / c.warps) + (float)c.share / (float)c.warps);
        const float cost = turns * ((float)(tiles * parts) + 0.22f * (float)mv) + (ls > 0 ? 2.2f : 0.f);
        if (!best.warps || cost < least) {
            best = c;
            least = cost;
        }
    }
    if (best.warps) return best;
    // more tiles than that: as many a block as fit, over several rounds of blocks
    for (int ls = 0; ls < end; ++ls)
        for (int tiles = std::min(most_tiles, ntiles); tiles >= 1; --tiles) {
            const W4Launch c = made(ls, tiles, (ntiles + tiles - 1) / tiles);
            if (c.smem <= kBlockSmem && (tiles >= 2 || ls == end - 1)) return c;
        }
    return W4Launch{};
}
// How often all SMs take a block.
inline int rounds_of(const W4Launch& c, const int at_once[4]) {
    const int most = std::max(1, at_once[c.log_split]);
    return (c.grid + most - 1) / most;
}
// Whether the plan with the sums in the activations' place saves a round of blocks.
inline bool saves_a_round(const W4Launch& in_act, const W4Launch& own, const int at_once[4]) {
    return in_act.warps && (!own.warps || rounds_of(in_act, at_once) < rounds_of(own, at_once));
}

// How many clusters of 1, 2, 4 and 8 blocks of a kernel run at once with a block an SM,
// the kernel's shared-memory limit raised; once per device.
template <int MV, int PARTS, bool IN_ACT>
cudaError_t prepare_gemv_w4(int dev, int sms, int at_once[4]) {
    static std::mutex mu;
    static int at_once_of[64][4] = {};
    const auto kern = gemv_w4_kernel<MV, PARTS, IN_ACT>;
    const std::lock_guard<std::mutex> lock(mu);
    int* v = at_once_of[dev & 63];
    if (!v[0]) {
        cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kBlockSmem);
        if (e != cudaSuccess) return e;
        int n[4] = {sms, 0, 0, 0};
        for (int ls = 1; ls < 4; ++ls) {
            e = clusters_at_once(kern, max_warps(MV) * 32, kBlockSmem, 1, 1 << ls, &n[ls]);
            if (e != cudaSuccess) return e;
        }
        std::copy(n, n + 4, v);
    }
    std::copy(v, v + 4, at_once);
    return cudaSuccess;
}

template <int MV, int PARTS>
cudaError_t launch_gemv_w4_as(const W4Params& p, int dev, int sms, cudaStream_t s) {
    int at_once[4];
    cudaError_t e = prepare_gemv_w4<MV, PARTS, false>(dev, sms, at_once);
    if (e != cudaSuccess) return e;
    const W4Launch c = plan_gemv_w4(p, MV, PARTS, false, at_once);
    if constexpr (has_in_act(MV, PARTS)) {
        int at_once_in[4];
        e = prepare_gemv_w4<MV, PARTS, true>(dev, sms, at_once_in);
        if (e != cudaSuccess) return e;
        const W4Launch in = plan_gemv_w4(p, MV, PARTS, true, at_once_in);
        if (saves_a_round(in, c, at_once))
            return launch_ordered(gemv_w4_kernel<MV, PARTS, true>, dim3(in.grid, 1, 1 << in.log_split), dim3(in.warps * 32),
                                  in.smem, s, 1, 1 << in.log_split, p, in);
    }
    if (!c.warps) return cudaErrorInvalidValue;
    return launch_ordered(gemv_w4_kernel<MV, PARTS, false>, dim3(c.grid, 1, 1 << c.log_split), dim3(c.warps * 32), c.smem, s,
                          1, 1 << c.log_split, p, c);
}

cudaError_t launch_gemv_w4(const W4Params& p, int dev, int sms, cudaStream_t s) {
    const bool two = p.epi == 2;
    if (p.M == 1) return two ? launch_gemv_w4_as<1, 2>(p, dev, sms, s) : launch_gemv_w4_as<1, 1>(p, dev, sms, s);
    if (p.M == 2) return two ? launch_gemv_w4_as<2, 2>(p, dev, sms, s) : launch_gemv_w4_as<2, 1>(p, dev, sms, s);
    if (p.M <= 4) return two ? launch_gemv_w4_as<4, 2>(p, dev, sms, s) : launch_gemv_w4_as<4, 1>(p, dev, sms, s);
    return two ? launch_gemv_w4_as<8, 2>(p, dev, sms, s) : launch_gemv_w4_as<8, 1>(p, dev, sms, s);
}

bool misaligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0; }

int report_w4(cudaError_t e, const char* what) {
    std::fprintf(stderr, "tts: %s failed: %s\n", what, cudaGetErrorString(e));
    return TTS_ERR_CUDA;
}

}  // namespace
}  // namespace tts

extern "C" int tts_quantize_w4_weight(const void* W, int N, int K, void* W4, void* s, void* stream) {
    using namespace tts;
    if (!W || !W4 || !s || N < 1 || K < 1 || K % kW4Group) return TTS_ERR_ARG;
    if (misaligned(W, 16) || misaligned(W4, 16) || misaligned(s, 4)) return TTS_ERR_ARG;
    const size_t groups = (size_t)N * (K / kW4Group);
    if (overwritten({{W4, groups * (kW4Group / 2)}, {s, groups * 2}}, {{W, groups * kW4Group * 2}})) return TTS_ERR_ARG;
    const size_t blocks = (groups + 7) / 8;
    if (blocks > 0x7fffffffu) return TTS_ERR_ARG;
    quantize_w4_kernel<<<(unsigned)blocks, 256, 0, static_cast<cudaStream_t>(stream)>>>(
        static_cast<const __nv_bfloat16*>(W), groups, static_cast<uint8_t*>(W4), static_cast<__nv_bfloat16*>(s));
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? TTS_OK : report_w4(e, "tts_quantize_w4_weight");
}

extern "C" int tts_gemv_w4(const float* x, const void* W4, const void* s, const float* resid, const void* gamma,
                           float* y, int M, int N, int K, int epi, float eps, void* stream) {
    using namespace tts;
    if (!x || !W4 || !s || !y || M < 1 || M > kW4MaxM || N < 1 || N > (1 << 24)) return TTS_ERR_ARG;
    if (K < kW4Group || K % kW4Group || K > kW4MaxK || epi < 0 || epi > 2) return TTS_ERR_ARG;
    if ((epi == 1) != (resid != nullptr)) return TTS_ERR_ARG;
    if (gamma && !(eps >= 0.f)) return TTS_ERR_ARG;
    if (misaligned(x, 16) || misaligned(W4, 16) || misaligned(s, 4) || misaligned(y, 4) || misaligned(resid, 4) ||
        misaligned(gamma, 16))
        return TTS_ERR_ARG;
    const size_t yb = sizeof(float) * (size_t)M * N, rows = (size_t)N * (epi == 2 ? 2 : 1);
    if (overwritten({{y, yb}}, {{x, sizeof(float) * (size_t)M * K},
                                {W4, rows * (K / 2)},
                                {s, rows * (K / kW4Group) * 2},
                                {gamma, 2 * (size_t)K},
                                {resid == y ? nullptr : resid, yb}}))
        return TTS_ERR_ARG;
    W4Params p{x, static_cast<const uint8_t*>(W4), static_cast<const __nv_bfloat16*>(s), resid,
               static_cast<const __nv_bfloat16*>(gamma), y, M, N, K, epi, eps};
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return TTS_ERR_CUDA;
    const cudaError_t e = launch_gemv_w4(p, dev, sms, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? TTS_OK : report_w4(e, "tts_gemv_w4");
}
