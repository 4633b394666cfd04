// Log probabilities of given codes, the entropy of the distribution and its
// top alternatives, from the head's logits (sm_103a).
#include <cmath>
#include <cstdio>

#include "kernels.h"
#include "tts_decode.h"

namespace tts {
namespace {

// Sort key of entry i: larger logits first, equal ones by the lower index
// (-0 equals +0; NaN below everything).
__device__ __forceinline__ unsigned long long top_key(float z, int i) {
    uint32_t b = __float_as_uint(z + 0.f);
    b = (b & 0x80000000u) ? ~b : b | 0x80000000u;
    if (isnan(z)) b = 0;
    return (unsigned long long)b << 32 | (uint32_t)~i;
}

// One block per (row, codebook): maximum, sums, then one search per alternative.
__global__ void __launch_bounds__(256) logprobs_kernel(const LogprobParams p) {
    __shared__ float red[32];
    __shared__ unsigned long long redk[8];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const size_t item = blockIdx.x;
    const int V = p.V;
    const float* z = p.logits + (item / p.n_cb) * p.ld + (item % p.n_cb) * V;
    float m = -INFINITY, is_nan = 0.f;
    for (int i = threadIdx.x; i < V; i += 256) {
        m = fmaxf(m, z[i]);
        if (isnan(z[i])) is_nan = 1.f;
    }
    m = block_max(m, red);
    const bool none = m == -INFINITY && block_max(is_nan, red) == 0.f;  // every entry is -inf
    float l = 0.f, w = 0.f;
    for (int i = threadIdx.x; i < V; i += 256) {
        const float d = z[i] - m, e = expf(d * p.inv_t);
        l += e;
        w += e > 0.f ? e * (d * p.inv_t) : 0.f;
    }
    l = block_sum(l, red);
    w = block_sum(w, red);
    const float logl = logf(l);
    if (threadIdx.x == 0) {
        if (p.logprob) {
            const int c = p.codes[item];
            p.logprob[item] = c < 0 || c >= V ? NAN : none ? -INFINITY : (z[c] - m) * p.inv_t - logl;
        }
        if (p.entropy) p.entropy[item] = none ? 0.f : logl - w / l;
    }
    unsigned long long last = ~0ull;
    for (int k = 0; k < p.top; ++k) {
        unsigned long long best = 0;
        for (int i = threadIdx.x; i < V; i += 256) {
            const unsigned long long key = top_key(z[i], i);
            if (key < last && key > best) best = key;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const unsigned long long other = __shfl_xor_sync(0xffffffffu, best, o);
            best = other > best ? other : best;
        }
        __syncthreads();
        if (lane == 0) redk[warp] = best;
        __syncthreads();
        for (int j = 0; j < 8; ++j) best = redk[j] > best ? redk[j] : best;
        last = best;
        if (threadIdx.x == 0) {
            const int c = (int)~(uint32_t)best;
            p.top_codes[item * p.top + k] = c;
            p.top_logprob[item * p.top + k] = none ? -INFINITY : (z[c] - m) * p.inv_t - logl;
        }
    }
}

}  // namespace

cudaError_t launch_logprobs(const LogprobParams& p, cudaStream_t s) {
    logprobs_kernel<<<(unsigned)((long long)p.rows * p.n_cb), 256, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace tts

extern "C" int tts_code_logprobs(const float* logits, long long ld, const int32_t* codes, int rows, int n_cb,
                                 int cb_vocab, float temperature, int top, float* logprob, float* entropy,
                                 int32_t* top_codes, float* top_logprob, void* stream) {
    using namespace tts;
    if (rows < 0 || n_cb < 1 || n_cb > kMaxCodebooks || cb_vocab < 2 || cb_vocab > (1 << 20)) return TTS_ERR_ARG;
    if (!logits || ld < (long long)n_cb * cb_vocab || top < 0 || top > kMaxTop || top > cb_vocab) return TTS_ERR_ARG;
    if ((long long)rows * n_cb > 0x7fffffffLL) return TTS_ERR_ARG;
    if (!(temperature > 0.f) || !std::isfinite(temperature) || !std::isfinite(1.f / temperature)) return TTS_ERR_ARG;
    if ((logprob != nullptr) != (codes != nullptr)) return TTS_ERR_ARG;
    if ((top > 0) != (top_codes != nullptr) || (top > 0) != (top_logprob != nullptr)) return TTS_ERR_ARG;
    const uintptr_t all = reinterpret_cast<uintptr_t>(logits) | reinterpret_cast<uintptr_t>(codes) |
                          reinterpret_cast<uintptr_t>(logprob) | reinterpret_cast<uintptr_t>(entropy) |
                          reinterpret_cast<uintptr_t>(top_codes) | reinterpret_cast<uintptr_t>(top_logprob);
    if (all & 3) return TTS_ERR_ARG;
    if (rows == 0) return TTS_OK;
    LogprobParams p{logits, ld, codes, rows, n_cb, cb_vocab, 1.f / temperature, top, logprob, entropy, top_codes,
                    top_logprob};
    const cudaError_t e = launch_logprobs(p, static_cast<cudaStream_t>(stream));
    if (e == cudaSuccess) return TTS_OK;
    std::fprintf(stderr, "tts: tts_code_logprobs failed: %s\n", cudaGetErrorString(e));
    return TTS_ERR_CUDA;
}
