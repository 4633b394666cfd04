// 4-bit weights with group scales: quantisation of a bf16 matrix and the
// matrix-vector product of a decode step (sm_103a).
//
// Format: W4 uint8 [N][K/2], low nibble = even k, u in 0..15; s bf16
// [N][K/128]; weight = s * (u - 8).
#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdio>

#include "kernels.h"
#include "tts_decode.h"

namespace tts {
namespace {

constexpr int kW4Group = 128;
constexpr int kW4MaxM = 8;
constexpr int kW4MaxK = 12288;

__device__ __forceinline__ void cp_async16_at(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// 4 bytes of which the last two may be left out (read as zero)
__device__ __forceinline__ void cp_async4_at(uint32_t dst, const void* src, int bytes) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit_group() { asm volatile("cp.async.commit_group;" ::: "memory"); }
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
// the weights once (at most 8 flops a byte), so everything else has to stay
// below that: a weight may cost about 2.7 of an SM's lane instructions.
//
// Codes are the A operand of m16n8k16 products (fp16, fp32 sums) as they lie
// in memory: a nibble masked out of its 16-bit half IS the fp16 subnormal
// u 2^-24, and a byte of two nibbles is (u + 16 u') 2^-24, exact, so a code
// costs half an instruction and no conversion; q u + q' u' = (q - q'/16) u +
// (q'/16)(u + 16 u') moves the rest to the activations.  These are the B
// operand: fp32, scaled per 128 group by a power of two to below 2^15 and split
// into two fp16 parts (22 bits, and 2^-39 of the group's largest), columns 2m and
// 2m + 1 for vector m, so up to four vectors cost what one does.  Group sums
// leave the tensor core once a group and are scaled and added in fp32:
// acc += s (2^24-e part - 8 sum(a)).
//
// A block takes tiles of 16 rows (epi 2: a gate and an up tile), about one block
// an SM; its warps take one slice of the groups each, the same for all its
// tiles, so a warp prepares its slice of the activations once and for itself.
// A lane copies exactly the 2 x 16 bytes of a group that it uses (rows r and
// r + 8, piece t), asynchronously into a ring of its own: no barrier before all
// of a block's tiles are done and the warps' sums are added.
// (Four small blocks an SM were measured first: gate/up at one vector took
// 11.7 us, most of it preparing the same activations four times.)
constexpr int kMaxTiles = 8;  // tiles (epi 2: pairs) a block, at most
constexpr int kStage = 1024 + 64;  // an item (tile, group): codes, then a word with each row's scale

struct W4Launch {
    int warps, tiles, slice;  // tiles a block and groups a warp, at most
    int grid;
    size_t smem;
};

__device__ __forceinline__ void mma16816_f16(float c[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                             uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Bytes 0 and 2 or 1 and 3 of w, each in the low byte of a 16-bit half.
__device__ __forceinline__ uint32_t even_bytes(uint32_t w) { return w & 0x00ff00ffu; }
__device__ __forceinline__ uint32_t odd_bytes(uint32_t w) { return __byte_perm(w, 0u, 0x4341u); }

// Shared memory of a warp: [ring][activations: slice x 4 words x 2 MV columns x
// 4 pieces x 16 bytes][per group and vector: (2^24 over its power of two, 8 sum)].
// Then the block's: [sums: tiles x parts x 16 rows x MV x warps][sums of squares].
__host__ __device__ constexpr int act_group_bytes(int mv) { return 4 * 2 * mv * 4 * 16; }
__host__ __device__ inline size_t warp_bytes(int mv, int ring, int slice) {
    return ((size_t)ring * kStage + (size_t)slice * (act_group_bytes(mv) + mv * 8) + 15) & ~(size_t)15;
}
__host__ __device__ constexpr int max_warps(int mv) { return mv == 4 ? 16 : 24; }

template <int MV, int PARTS, int RING>  // vectors a block (1, 2, 4), tiles an output tile takes, items in flight a warp
__global__ void __launch_bounds__(max_warps(MV) * 32, 1) gemv_w4_kernel(const W4Params p, const W4Launch c) {
    extern __shared__ __align__(128) uint8_t smem[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, W = c.warps;
    const int r = lane >> 2, t = lane & 3;
    const int groups = p.K / kW4Group;
    const int g0 = groups * warp / W, ng = groups * (warp + 1) / W - g0;  // at least 1: W <= groups
    const int m0 = blockIdx.y * MV, mv = min(MV, p.M - m0);
    const int ntiles = (p.N + 15) / 16;
    const int tile0 = blockIdx.x, step = gridDim.x;
    const int nt = (ntiles - tile0 + step - 1) / step;  // this block's tiles: tile0, tile0 + step, ...

    uint8_t* mine = smem + (size_t)warp * warp_bytes(MV, RING, c.slice);
    uint8_t* act = mine + RING * kStage;
    float2* act_par = reinterpret_cast<float2*>(act + c.slice * act_group_bytes(MV));
    float* sums = reinterpret_cast<float*>(smem + (size_t)W * warp_bytes(MV, RING, c.slice));
    float* sq = sums + (size_t)c.tiles * PARTS * 16 * MV * W;  // [MV][W]

    // ---- activations of the slice's first group: before the copies, which would
    // hold them up
    float4 xs[MV];
    uint2 gb = {};
    auto load_x = [&](int g) {
        const size_t k = (size_t)(g0 + g) * kW4Group + 4 * lane;
#pragma unroll
        for (int m = 0; m < MV; ++m)
            xs[m] = m < mv ? *reinterpret_cast<const float4*>(p.x + (size_t)(m0 + m) * p.K + k) : make_float4(0.f, 0.f, 0.f, 0.f);
        if (p.gamma) gb = *reinterpret_cast<const uint2*>(p.gamma + k);
    };
    load_x(0);

    // ---- copies, item by item: tile, part of it, group
    const uint32_t ring = smem_u32(mine);
    const long long total = (long long)p.N * PARTS * groups;  // scales in all
    int iq = 0, ig = 0;                                       // next item to copy
    const uint8_t *pa = nullptr, *pb = nullptr;
    long long ps = 0;
    // row i of the block's tile q; past the end the last row, whose result is not
    // stored
    auto row_of = [&](int q, int i) {
        const int tile = tile0 + (q / PARTS) * step;
        return min(tile * 16 + i, p.N - 1) + (q % PARTS) * p.N;
    };
    auto issue = [&](int stage) {
        if (iq >= nt * PARTS) return;
        if (ig == 0) {
            pa = p.W4 + (size_t)row_of(iq, r) * (p.K / 2) + (size_t)g0 * 64 + t * 16;
            pb = p.W4 + (size_t)row_of(iq, r + 8) * (p.K / 2) + (size_t)g0 * 64 + t * 16;
            ps = (long long)row_of(iq, lane & 15) * groups + g0;
        }
        const uint32_t dst = ring + stage * kStage;
        cp_async16_at(dst + lane * 16, pa + ig * 64);
        cp_async16_at(dst + 512 + lane * 16, pb + ig * 64);
        // the 4-byte word that holds the row's scale; the last one of all may be
        // half a word
        const long long at = (ps + ig) & ~1ll;
        if (lane < 16) cp_async4_at(dst + 1024 + lane * 4, p.s + at, at + 1 < total ? 4 : 2);
        if (++ig == ng) {
            ig = 0;
            ++iq;
        }
    };
#pragma unroll
    for (int i = 0; i < RING - 1; ++i) {
        issue(i);
        cp_async_commit_group();
    }

    // half-warp h of the block adds up output h, h + 2 W, ... at the end: what it
    // adds the first of them to
    const int half = threadIdx.x >> 4, h_lane = threadIdx.x & 15;
    auto place = [&](int i, size_t* at) {  // output i: (tile, row, vector)
        const int n = (tile0 + i / (16 * MV) * step) * 16 + (i / MV) % 16, m = i % MV;
        *at = (size_t)(m0 + m) * p.N + n;
        return i < nt * 16 * MV && n < p.N && m < mv;
    };
    float resid = 0.f;
    if (p.resid && h_lane == 0) {
        size_t at;
        if (place(half, &at)) resid = p.resid[at];
    }

    // ---- this warp's slice of the activations
    float ss[MV];
#pragma unroll
    for (int m = 0; m < MV; ++m) ss[m] = 0.f;
    for (int g = 0; g < ng; ++g) {
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
        if (g + 1 < ng) load_x(g + 1);
        uint8_t* dst = act + (size_t)g * act_group_bytes(MV) + ((lane >> 1) & 3) * (2 * MV * 64) + (lane >> 3) * 16 + (lane & 1) * 8;
#pragma unroll
        for (int m = 0; m < MV; ++m) {
            const float sum = warp_sum((a[m][0] + a[m][1]) + (a[m][2] + a[m][3]));
            const uint32_t amax = __reduce_max_sync(
                0xffffffffu,
                __float_as_uint(fmaxf(fmaxf(fabsf(a[m][0]), fabsf(a[m][1])), fmaxf(fabsf(a[m][2]), fabsf(a[m][3])))));
            // the group's power of two: largest to [2^14, 2^15)
            const int e = max((int)(amax >> 23), 14);
            const float f = __uint_as_float((uint32_t)(268 - e) << 23);
            if (lane == 0) act_par[g * MV + m] = make_float2(__uint_as_float((uint32_t)min(10 + e, 254) << 23), 8.f * sum);
            // channels 4 l .. 4 l + 3 are nibbles 4 (l % 2) + 0..3 of word (l / 2) % 4 of
            // piece l / 8: of the pairs (0, 4), (1, 5), (2, 6), (3, 7) an even lane
            // has the low halves, an odd lane the high ones
            uint32_t hi[2], lo[2];  // (pair 0, pair 1), (pair 2, pair 3)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const float v0 = (a[m][2 * j] - 0.0625f * a[m][2 * j + 1]) * f, v1 = 0.0625f * a[m][2 * j + 1] * f;
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
            *reinterpret_cast<uint2*>(dst + 2 * m * 64) = make_uint2(__byte_perm(eh, oh, 0x5410), __byte_perm(eh, oh, 0x7632));
            *reinterpret_cast<uint2*>(dst + 2 * m * 64 + 64) = make_uint2(__byte_perm(el, ol, 0x5410), __byte_perm(el, ol, 0x7632));
        }
    }
    if (p.gamma) {
#pragma unroll
        for (int m = 0; m < MV; ++m) {
            ss[m] = warp_sum(ss[m]);
            if (lane == 0) sq[m * W + warp] = ss[m];
        }
    }
    __syncwarp();

    // ---- the products
    int stage = 0, fill = RING - 1;
    const bool column = r < 2 * MV;
    const uint8_t* my_act = act + r * 64 + t * 16;
    for (int q = 0; q < nt * PARTS; ++q) {
        float acc[2] = {0.f, 0.f};
        // which half of its word a row's first scale is
        const int oa = (row_of(q, r) & groups & 1) ^ (g0 & 1), ob = (row_of(q, r + 8) & groups & 1) ^ (g0 & 1);
        for (int g = 0; g < ng; ++g) {
            asm volatile("cp.async.wait_group %0;" ::"n"(RING - 2) : "memory");
            __syncwarp();  // the scales come through other lanes' copies
            issue(fill);
            cp_async_commit_group();
            if (++fill == RING) fill = 0;
            const uint8_t* st = mine + stage * kStage;
            if (++stage == RING) stage = 0;
            const uint4 wa = *reinterpret_cast<const uint4*>(st + lane * 16);
            const uint4 wb = *reinterpret_cast<const uint4*>(st + 512 + lane * 16);
            const uint32_t sa = *reinterpret_cast<const uint32_t*>(st + 1024 + r * 4);
            const uint32_t sb = *reinterpret_cast<const uint32_t*>(st + 1024 + r * 4 + 32);
            const uint32_t ua[4] = {wa.x, wa.y, wa.z, wa.w}, ub[4] = {wb.x, wb.y, wb.z, wb.w};
            float d[2][4] = {};
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                uint4 b = make_uint4(0, 0, 0, 0);
                if (column) b = *reinterpret_cast<const uint4*>(my_act + (size_t)g * act_group_bytes(MV) + w * (2 * MV * 64));
                const uint32_t x0 = even_bytes(ua[w]), y0 = even_bytes(ub[w]), x1 = odd_bytes(ua[w]), y1 = odd_bytes(ub[w]);
                mma16816_f16(d[0], x0 & 0x000f000fu, y0 & 0x000f000fu, x0, y0, b.x, b.y);
                mma16816_f16(d[1], x1 & 0x000f000fu, y1 & 0x000f000fu, x1, y1, b.z, b.w);
            }
            const float2 ap = act_par[g * MV + (t < MV ? t : 0)];
            const float va = (d[0][0] + d[1][0]) + (d[0][1] + d[1][1]), vb = (d[0][2] + d[1][2]) + (d[0][3] + d[1][3]);
            acc[0] = fmaf((g ^ oa) & 1 ? bf16hi(sa) : bf16lo(sa), fmaf(va, ap.x, -ap.y), acc[0]);
            acc[1] = fmaf((g ^ ob) & 1 ? bf16hi(sb) : bf16lo(sb), fmaf(vb, ap.x, -ap.y), acc[1]);
        }
        if (t < MV) {
            float* s = sums + (size_t)(q * 16 * MV + t) * W + warp;
            s[(size_t)r * MV * W] = acc[0];
            s[(size_t)(r + 8) * MV * W] = acc[1];
        }
    }
    __syncthreads();

    // ---- the warps' sums, an output a half-warp, and the epilogue
    auto half_sum = [&](const float* v) {  // of W values, in a fixed order
        float s = h_lane < W ? v[h_lane] : 0.f;
        if (h_lane + 16 < W) s += v[h_lane + 16];
#pragma unroll
        for (int d = 8; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
        return s;
    };
    const int outs = nt * 16 * MV;
    for (int i0 = 0; i0 < outs; i0 += 2 * W) {
        const int i = i0 + half, at_i = min(i, outs - 1);
        const int q = at_i / (16 * MV), rest = at_i % (16 * MV);
        float v[PARTS], rms = 1.f;
#pragma unroll
        for (int h = 0; h < PARTS; ++h) v[h] = half_sum(sums + (size_t)((q * PARTS + h) * 16 * MV + rest) * W);
        if (p.gamma) rms = 1.f / sqrtf(half_sum(sq + (at_i % MV) * W) / (float)p.K + p.eps);
        size_t at;
        if (place(i, &at) && h_lane == 0) {
            float y = v[0] * rms;
            if (p.resid) y += i0 == 0 ? resid : p.resid[at];
            if (PARTS == 2) y = y / (1.f + expf(-y)) * (v[PARTS - 1] * rms);
            p.y[at] = y;
        }
    }
}

constexpr size_t kBlockSmem = 227 * 1024;

// Blocks, warps a block and tiles a block for p at MV vectors a block; ring is
// set to the copies in flight a warp.
W4Launch plan_gemv_w4(const W4Params& p, int mv, int parts, int ny, int sms, int* ring) {
    const int groups = p.K / kW4Group, ntiles = (p.N + 15) / 16;
    // a block an SM, which takes its tiles one after another
    int grid = std::min(ntiles, std::max(1, sms / ny));
    grid = std::max(grid, (ntiles + kMaxTiles - 1) / kMaxTiles);
    const int tiles = (ntiles + grid - 1) / grid;
    W4Launch best{};
    int best_cost = 1 << 30;
    for (const int rg : {8, 3})
        for (int w = std::min(groups, max_warps(mv)); w >= 1; --w) {
            const int slice = (groups + w - 1) / w;
            const size_t smem = w * warp_bytes(mv, rg, slice) + 4 * (size_t)w * mv * (tiles * parts * 16 + 1);
            if (smem > kBlockSmem) continue;
            // items of a tile that the fullest scheduler issues; under 12 warps
            // they wait for one another more
            const int cost = (w + 3) / 4 * slice * (w >= 12 ? 4 : 5);
            if (cost < best_cost) {
                best_cost = cost;
                best = W4Launch{w, tiles, slice, grid, smem};
                *ring = rg;
            }
        }
    return best;
}

template <int MV, int PARTS, int RING>
cudaError_t launch_gemv_w4_as(const W4Params& p, const W4Launch& c, int ny, int dev, cudaStream_t s) {
    static std::atomic<unsigned long long> ready{0};  // devices whose shared-memory limit is raised
    const unsigned long long bit = 1ull << (dev & 63);
    const auto kern = gemv_w4_kernel<MV, PARTS, RING>;
    if (!(ready.load(std::memory_order_relaxed) & bit)) {
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kBlockSmem);
        if (e != cudaSuccess) return e;
        ready.fetch_or(bit, std::memory_order_relaxed);
    }
    kern<<<dim3(c.grid, ny), c.warps * 32, c.smem, s>>>(p, c);
    return cudaGetLastError();
}

template <int MV>
cudaError_t launch_gemv_w4_mv(const W4Params& p, int dev, int sms, cudaStream_t s) {
    const int ny = (p.M + MV - 1) / MV;
    int ring = 0;
    const W4Launch c = plan_gemv_w4(p, MV, p.epi == 2 ? 2 : 1, ny, sms, &ring);
    if (!c.warps) return cudaErrorInvalidValue;
    if (p.epi == 2)
        return ring == 8 ? launch_gemv_w4_as<MV, 2, 8>(p, c, ny, dev, s) : launch_gemv_w4_as<MV, 2, 3>(p, c, ny, dev, s);
    return ring == 8 ? launch_gemv_w4_as<MV, 1, 8>(p, c, ny, dev, s) : launch_gemv_w4_as<MV, 1, 3>(p, c, ny, dev, s);
}

cudaError_t launch_gemv_w4(const W4Params& p, int dev, int sms, cudaStream_t s) {
    if (p.M == 1) return launch_gemv_w4_mv<1>(p, dev, sms, s);
    if (p.M == 2) return launch_gemv_w4_mv<2>(p, dev, sms, s);
    return launch_gemv_w4_mv<4>(p, dev, sms, s);
}

bool overlap(const void* a, size_t na, const void* b, size_t nb) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + nb && y < x + na;
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
    // other blocks still read the inputs while the first ones write y
    if (overlap(y, yb, x, sizeof(float) * (size_t)M * K) || overlap(y, yb, W4, rows * (K / 2)) ||
        overlap(y, yb, s, rows * (K / kW4Group) * 2) || (gamma && overlap(y, yb, gamma, 2 * (size_t)K)) ||
        (resid && resid != y && overlap(y, yb, resid, yb)))
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
