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
// A block takes tiles of 16 rows (epi 2: a gate and an up tile), its warps one
// slice of the groups each, the same for all its tiles, so a warp prepares its
// slice of the activations once, for itself.  A lane copies exactly the 2 x 16
// bytes a group that it uses (row r and r + 8, piece t), asynchronously into a
// ring of its own: no barrier before a block's tiles are summed.
constexpr int kMaxWarps = 16;
constexpr int kRing = 4;      // items (tile, group) in flight a warp, 1 KB each
constexpr int kMaxTiles = 8;  // tiles (epi 2: pairs) a block, at most

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
// 4 pieces x 16 bytes][per group and vector: (2^24 over its power of two, 8 sum)]
// [scales: tiles x 16 rows x the 4-byte words that cover a slice].
__host__ __device__ inline int act_group_bytes(int mv) { return 4 * 2 * mv * 4 * 16; }
__host__ __device__ inline int scale_words(int slice) { return slice / 2 + 1; }
__host__ __device__ inline size_t warp_bytes(int mv, int slice, int tiles) {
    const size_t b = (size_t)kRing * 1024 + (size_t)slice * act_group_bytes(mv) + (size_t)slice * mv * 8 +
                     (size_t)tiles * 16 * scale_words(slice) * 4;
    return (b + 15) & ~(size_t)15;
}

template <int MV>  // vectors of this block: 1, 2 or 4 columns pairs
__global__ void __launch_bounds__(kMaxWarps * 32, MV == 1 ? 2 : 1) gemv_w4_kernel(const W4Params p, const W4Launch c) {
    extern __shared__ __align__(128) uint8_t smem[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, W = c.warps;
    const int r = lane >> 2, t = lane & 3;
    const int groups = p.K / kW4Group, parts = p.epi == 2 ? 2 : 1;
    const int g0 = (int)((long long)groups * warp / W), ng = (int)((long long)groups * (warp + 1) / W) - g0;
    const int m0 = blockIdx.y * MV, mv = min(MV, p.M - m0);
    const int ntiles = (p.N + 15) / 16;
    const int tile0 = blockIdx.x, step = gridDim.x;
    const int nt = (ntiles - tile0 + step - 1) / step;  // this block's tiles: tile0, tile0 + step, ...
    const int rows_total = p.N * parts;

    uint8_t* mine = smem + (size_t)warp * warp_bytes(MV, c.slice, c.tiles * parts);
    uint8_t* act = mine + kRing * 1024;
    float2* act_par = reinterpret_cast<float2*>(act + c.slice * act_group_bytes(MV));
    uint32_t* scl = reinterpret_cast<uint32_t*>(act_par + c.slice * MV);
    float* sums = reinterpret_cast<float*>(smem + (size_t)W * warp_bytes(MV, c.slice, c.tiles * parts));
    float* sq = sums + (size_t)c.tiles * parts * W * 16 * MV;  // [W][MV] sums of squares

    // row of the weights that row i of tile q = (tile, part) is; past the end, the
    // last one (its result is not stored)
    auto row_of = [&](int q, int i) {
        const int tile = tile0 + (q / parts) * step;
        return min(tile * 16 + i, p.N - 1) + (q % parts) * p.N;
    };
    const int items = nt * parts * ng;
    const uint32_t ring = smem_u32(mine) + lane * 16;
    int iq = 0, ig = 0;  // next item to copy
    const uint8_t *pa = nullptr, *pb = nullptr;
    auto issue = [&](int stage) {
        if (ig == 0) {
            pa = p.W4 + (size_t)row_of(iq, r) * (p.K / 2) + (size_t)g0 * 64 + t * 16;
            pb = p.W4 + (size_t)row_of(iq, r + 8) * (p.K / 2) + (size_t)g0 * 64 + t * 16;
        }
        cp_async16_at(ring + stage * 1024, pa + ig * 64);
        cp_async16_at(ring + stage * 1024 + 512, pb + ig * 64);
        if (++ig == ng) { ig = 0; ++iq; }
    };
    int issued = 0;
    // scales of all tiles first: 4-byte words that cover each row's slice
    const int sw = scale_words(c.slice);
    if (ng > 0) {
        const long long total = (long long)rows_total * groups;  // scales in all
        for (int i = lane; i < nt * parts * 16 * sw; i += 32) {
            const int row = row_of(i / (16 * sw), (i / sw) & 15), wd = i % sw;
            const long long at = ((long long)row * groups + g0) / 2 * 2 + 2 * wd;
            if (at < (long long)row * groups + g0 + ng)
                cp_async4_at(smem_u32(scl + i), p.s + at, at + 1 < total ? 4 : 2);
        }
    }
    cp_async_commit_group();
    for (; issued < kRing - 1; ++issued) {
        if (issued < items) issue(issued);
        cp_async_commit_group();
    }

    // ---- this warp's slice of the activations
    float ss[MV];
#pragma unroll
    for (int m = 0; m < MV; ++m) ss[m] = 0.f;
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
    for (int g = 0; g < ng; ++g) {
        float4 x4[MV];
#pragma unroll
        for (int m = 0; m < MV; ++m) x4[m] = xs[m];
        float gm[4] = {1.f, 1.f, 1.f, 1.f};
        if (p.gamma) {
            gm[0] = bf16lo(gb.x);
            gm[1] = bf16hi(gb.x);
            gm[2] = bf16lo(gb.y);
            gm[3] = bf16hi(gb.y);
        }
        if (g + 1 < ng) load_x(g + 1);
#pragma unroll
        for (int m = 0; m < MV; ++m) {
            float a[4] = {x4[m].x, x4[m].y, x4[m].z, x4[m].w};
            if (p.gamma) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    ss[m] = fmaf(a[j], a[j], ss[m]);
                    a[j] *= gm[j];
                }
            }
            const float sum = warp_sum((a[0] + a[1]) + (a[2] + a[3]));
            const uint32_t amax = __reduce_max_sync(
                0xffffffffu, __float_as_uint(fmaxf(fmaxf(fabsf(a[0]), fabsf(a[1])), fmaxf(fabsf(a[2]), fabsf(a[3])))));
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
                const float v0 = (a[2 * j] - 0.0625f * a[2 * j + 1]) * f, v1 = 0.0625f * a[2 * j + 1] * f;
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
            uint8_t* dst = act + (size_t)g * act_group_bytes(MV) + ((lane >> 1) & 3) * (2 * MV * 64) + 2 * m * 64 + (lane >> 3) * 16 +
                           (odd ? 8 : 0);
            *reinterpret_cast<uint2*>(dst) = make_uint2(__byte_perm(eh, oh, 0x5410), __byte_perm(eh, oh, 0x7632));
            *reinterpret_cast<uint2*>(dst + 64) = make_uint2(__byte_perm(el, ol, 0x5410), __byte_perm(el, ol, 0x7632));
        }
    }
    if (p.gamma) {
#pragma unroll
        for (int m = 0; m < MV; ++m) {
            ss[m] = warp_sum(ss[m]);
            if (lane == 0) sq[warp * MV + m] = ss[m];
        }
    }
    __syncwarp();

    // ---- the products: items (tile, group) in order
    int stage = 0, fill = kRing - 1;
    const bool column = r < 2 * MV;
    const uint8_t* my_act = act + r * 64 + t * 16;
    for (int q = 0; q < nt * parts; ++q) {
        float acc[2] = {0.f, 0.f};
        const long long ra = (long long)row_of(q, r) * groups + g0, rb = (long long)row_of(q, r + 8) * groups + g0;
        const uint16_t* sa = reinterpret_cast<const uint16_t*>(scl + (q * 16 + r) * sw) + (ra & 1);
        const uint16_t* sb = reinterpret_cast<const uint16_t*>(scl + (q * 16 + r + 8) * sw) + (rb & 1);
        for (int g = 0; g < ng; ++g) {
            asm volatile("cp.async.wait_group %0;" ::"n"(kRing - 2) : "memory");
            __syncwarp();  // the scales come through other lanes' copies
            if (issued < items) issue(fill);
            ++issued;
            cp_async_commit_group();
            if (++fill == kRing) fill = 0;
            const uint4 wa = *reinterpret_cast<const uint4*>(mine + stage * 1024 + lane * 16);
            const uint4 wb = *reinterpret_cast<const uint4*>(mine + stage * 1024 + 512 + lane * 16);
            if (++stage == kRing) stage = 0;
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
            acc[0] = fmaf(bf16_bits_to_f32(sa[g]), fmaf(va, ap.x, -ap.y), acc[0]);
            acc[1] = fmaf(bf16_bits_to_f32(sb[g]), fmaf(vb, ap.x, -ap.y), acc[1]);
        }
        if (t < MV) {
            float* s = sums + ((size_t)q * W + warp) * 16 * MV;
            s[r * MV + t] = acc[0];
            s[(r + 8) * MV + t] = acc[1];
        }
    }
    cp_async_wait_all();
    __syncthreads();

    // ---- the warps' sums, in order, and the epilogue
    for (int i = threadIdx.x; i < nt * 16 * MV; i += W * 32) {
        const int q = i / (16 * MV), row = (i / MV) & 15, m = i % MV;
        const int n = (tile0 + q * step) * 16 + row;
        if (n >= p.N || m >= mv) continue;
        float v[2] = {0.f, 0.f};
        for (int h = 0; h < parts; ++h)
            for (int w = 0; w < W; ++w) v[h] += sums[((size_t)(q * parts + h) * W + w) * 16 * MV + row * MV + m];
        if (p.gamma) {
            float s2 = 0.f;
            for (int w = 0; w < W; ++w) s2 += sq[w * MV + m];
            const float rms = 1.f / sqrtf(s2 / (float)p.K + p.eps);
            v[0] *= rms;
            v[1] *= rms;
        }
        const size_t at = (size_t)(m0 + m) * p.N + n;
        float y = v[0];
        if (p.epi == 1) y += p.resid[at];
        if (p.epi == 2) y = y / (1.f + expf(-y)) * v[1];
        p.y[at] = y;
    }
}

constexpr size_t kBlockSmem = 227 * 1024;

// Tiles a block, warps a block and shared memory for p at MV vectors a block.
W4Launch plan_gemv_w4(const W4Params& p, int mv, int ny, int sms) {
    const int groups = p.K / kW4Group, parts = p.epi == 2 ? 2 : 1, ntiles = (p.N + 15) / 16;
    W4Launch best{};
    // blocks that an SM gets of this many tiles, and the warps of each that make
    // about 24 an SM (enough copies in flight to cover the memory's latency)
    const int per_sm = std::max(1, std::min(6, (ntiles * ny + sms / 2) / sms));
    const int most = std::min(groups, std::max(4, std::min(kMaxWarps, 24 / per_sm)));
    // of the warp counts down to half of that, the one that leaves the fewest idle
    int warps = most;
    for (int w = most; w >= (most + 1) / 2; --w)
        if ((groups + w - 1) / w * w < (groups + warps - 1) / warps * warps) warps = w;
    for (;; --warps) {
        const int slice = (groups + warps - 1) / warps;
        // a tile a block while the SMs hold all blocks at once, then as many tiles
        // as it takes, for the activations are prepared once a block
        for (int tiles = 1; tiles <= kMaxTiles; ++tiles) {
            const size_t smem = warps * warp_bytes(mv, slice, tiles * parts) +
                                4 * ((size_t)tiles * parts * warps * 16 * mv + (size_t)warps * mv);
            if (smem > kBlockSmem) break;
            best = W4Launch{warps, tiles, slice, (ntiles + tiles - 1) / tiles, smem};
            // by shared memory and by registers (64, 92 and 110 a thread)
            const int by_regs = (mv == 1 ? 32 : mv == 2 ? 20 : 16) / warps;
            const int resident = std::max(1, std::min((int)(kBlockSmem / (smem + 1024)), by_regs));
            if ((long long)best.grid * ny <= (long long)resident * sms) return best;
        }
        if (best.warps || warps == 1) return best;
    }
}

template <int MV>
cudaError_t launch_gemv_w4_mv(const W4Params& p, int dev, int sms, cudaStream_t s) {
    static std::atomic<unsigned long long> ready{0};  // devices whose shared-memory limit is raised
    const unsigned long long bit = 1ull << (dev & 63);
    if (!(ready.load(std::memory_order_relaxed) & bit)) {
        const cudaError_t e =
            cudaFuncSetAttribute(gemv_w4_kernel<MV>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kBlockSmem);
        if (e != cudaSuccess) return e;
        ready.fetch_or(bit, std::memory_order_relaxed);
    }
    const int ny = (p.M + MV - 1) / MV;
    const W4Launch c = plan_gemv_w4(p, MV, ny, sms);
    if (!c.warps) return cudaErrorInvalidValue;
    gemv_w4_kernel<MV><<<dim3(c.grid, ny), c.warps * 32, c.smem, s>>>(p, c);
    return cudaGetLastError();
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
