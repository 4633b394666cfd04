// What the 4-bit decode operators and the code scoring share (sm_103a).
#pragma once

#include "common.cuh"

namespace tts {

// Launch with a programmatic edge from the kernel before it in the stream.
// The kernel triggers at its start and waits before its first access to global
// memory, so its blocks may start as soon as an SM is free while every memory
// access stays in stream order.  Its loads are ordinary ones: the read-only path
// wants memory that nobody writes while the kernel runs, its wait included.
// Clusters of cluster_y x cluster_z blocks.
template <typename... KArgs, typename... Args>
inline cudaError_t launch_ordered(void (*kern)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t s, int cluster_y,
                                  int cluster_z, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = 1;
    at[1].val.clusterDim.y = cluster_y;
    at[1].val.clusterDim.z = cluster_z;
    cfg.attrs = at;
    cfg.numAttrs = cluster_y * cluster_z > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, args...);
}

// How many clusters of cluster_y x cluster_z such blocks run at once (a cluster
// stays within a group of SMs, so fewer than SMs / blocks).
template <typename Kernel>
inline cudaError_t clusters_at_once(Kernel kern, int threads, size_t smem, int cluster_y, int cluster_z, int* n) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(1, cluster_y, cluster_z);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = 1;
    at[0].val.clusterDim.y = cluster_y;
    at[0].val.clusterDim.z = cluster_z;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaOccupancyMaxActiveClusters(n, kern, &cfg);
}

// Memory of a call's arguments (p may be null), and whether anything that the call
// writes lies over something else of it: other blocks still read what the first ones
// to finish would write.
struct Span {
    const void* p;
    size_t n;
};
inline bool overlap(const Span& a, const Span& b) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    return a.p && b.p && x < y + b.n && y < x + a.n;
}
template <size_t W, size_t R>
inline bool overwritten(const Span (&written)[W], const Span (&read)[R]) {
    for (size_t i = 0; i < W; ++i) {
        for (const Span& r : read)
            if (overlap(written[i], r)) return true;
        for (size_t j = 0; j < i; ++j)
            if (overlap(written[i], written[j])) return true;
    }
    return false;
}

// Whether the first phase of a barrier is over, its copies there.  A wait's limit is
// wall time, which also passes while the GPU is another process's: one that ran out
// is made once more before the copies count as lost (on their way they take
// microseconds).
__device__ __forceinline__ bool mbar_arrived(uint64_t* bar) {
    if (mbar_try_wait(bar, 0)) return true;
    uint64_t t0 = globaltimer_ns();
    bool again = true;
    while (!mbar_try_wait(bar, 0)) {
        if (globaltimer_ns() - t0 > kWaitLimitNs) {
            if (!again) return false;
            again = false;
            t0 = globaltimer_ns();
        }
    }
    return true;
}

// 4-bit codes as operands of fp16 products.  Each 16-bit half of w holds two bytes of
// two codes: nibble_bytes takes byte 0 of both halves (odd = 0) or byte 1 to the
// low byte of a half under 0x64, which reads as the fp16 value 1024 + byte.
// low_code and both_codes take the bias and the codes' centre away: u - 8 of the
// low code u, and (u - 8) + 16 (u' - 8) of the byte, exact and normal fp16.
// (Without the bias the codes are exact fp16 subnormals and cost no subtraction,
// but the tensor core aligns products by their exponent fields: sums then kept 18
// bits, measured, not 23.)
__device__ __forceinline__ uint32_t nibble_bytes(uint32_t w, int odd) {
    return odd ? __byte_perm(w, 0x64646464u, 0x4341u) : (w & 0x00ff00ffu) | 0x64006400u;
}
__device__ __forceinline__ uint32_t minus_half2(uint32_t x, uint32_t bias) {
    const __half2 r = __hsub2(*reinterpret_cast<const __half2*>(&x), *reinterpret_cast<const __half2*>(&bias));
    return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t low_code(uint32_t bytes, uint32_t bias = 0x64086408u) {
    return minus_half2(bytes & 0xff0fff0fu, bias);
}
__device__ __forceinline__ uint32_t both_codes(uint32_t bytes, uint32_t bias = 0x64886488u) {
    return minus_half2(bytes, bias);
}

// Pairs of fp32 in a 64-bit register: two lanes of arithmetic an instruction.
typedef unsigned long long f32x2;
__device__ __forceinline__ f32x2 pack2(float x, float y) {
    f32x2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ float2 unpack2(f32x2 v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
    f32x2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

// Log probabilities of given codes, entropy and top alternatives (logprobs.cu).
constexpr int kMaxTop = 32;  // alternatives per codebook, at most
struct LogprobParams {
    const float* logits;  // row r, codebook k at logits + r * ld + k * V
    long long ld;
    const int* codes;     // [rows][n_cb], or null
    int rows, n_cb, V;
    float two_over_t;     // 2 / temperature
    int top;
    float* logprob;       // [rows][n_cb], or null
    float* entropy;       // [rows][n_cb], or null
    int* top_codes;       // [rows][n_cb][top]
    float* top_logprob;
};
cudaError_t launch_logprobs(const LogprobParams& p, cudaStream_t s);

}  // namespace tts
