// 4-bit weights with group scales: quantisation of a bf16 matrix and the
// matrix-vector product of a decode step (sm_103a).
//
// Format: W4 uint8 [N][K/2], low nibble = even k, u in 0..15; s bf16
// [N][K/128]; weight = s * (u - 8).
#include <cmath>
#include <cstdio>

#include "kernels.h"
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

// One warp per output: every lane takes 8 consecutive k of every 256.
__global__ void __launch_bounds__(256) gemv_w4_kernel(const W4Params p) {
    const int lane = threadIdx.x & 31;
    const int n = blockIdx.x * 8 + (threadIdx.x >> 5);
    if (n >= p.N) return;
    const int parts = p.epi == 2 ? 2 : 1;
    for (int m = 0; m < p.M; ++m) {
        const float* x = p.x + (size_t)m * p.K;
        float r = 1.f;
        if (p.gamma) {
            float ss = 0.f;
            for (int k = lane; k < p.K; k += 32) ss += x[k] * x[k];
            r = 1.f / sqrtf(warp_sum(ss) / (float)p.K + p.eps);
        }
        float acc[2] = {0.f, 0.f};
        for (int h = 0; h < parts; ++h) {
            const size_t row = (size_t)n + (size_t)h * p.N;
            const uint8_t* w = p.W4 + row * (p.K / 2);
            const __nv_bfloat16* s = p.s + row * (p.K / kW4Group);
            for (int k = 8 * lane; k < p.K; k += 256) {
                const uint32_t q = *reinterpret_cast<const uint32_t*>(w + k / 2);
                float part = 0.f;
                for (int j = 0; j < 8; ++j) {
                    const float xv = p.gamma ? x[k + j] * __bfloat162float(p.gamma[k + j]) : x[k + j];
                    part = fmaf((float)((int)((q >> (4 * j)) & 15) - 8), xv, part);
                }
                acc[h] = fmaf(part, __bfloat162float(s[k / kW4Group]), acc[h]);
            }
            acc[h] = warp_sum(acc[h]) * r;
        }
        if (lane == 0) {
            const size_t at = (size_t)m * p.N + n;
            float v = acc[0];
            if (p.epi == 1) v += p.resid[at];
            if (p.epi == 2) v = v / (1.f + __expf(-v)) * acc[1];
            p.y[at] = v;
        }
    }
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
    if (misaligned(W, 16) || misaligned(W4, 16) || misaligned(s, 2)) return TTS_ERR_ARG;
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
    if (misaligned(x, 16) || misaligned(W4, 16) || misaligned(s, 2) || misaligned(y, 4) || misaligned(resid, 4) ||
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
    gemv_w4_kernel<<<(N + 7) / 8, 256, 0, static_cast<cudaStream_t>(stream)>>>(p);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? TTS_OK : report_w4(e, "tts_gemv_w4");
}
