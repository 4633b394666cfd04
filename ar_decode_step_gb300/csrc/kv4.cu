// A key-value cache held in 4 bits: writing bf16 rows in, reading them back,
// and the decode attention that reads it (sm_103a).
//
// A row of 128 channels is two halves of 64.  Half h has a bf16 minimum m and
// a bf16 scale s = bf16((max - m) / 15); a code u = clamp(rint((x - m) / s),
// 0, 15) stands for m + s u.  Byte 8r + j of the row's 64 holds channels
// 8r + 2j (low nibble) and 8r + 2j + 1 for j < 4, and the same channels + 64
// in byte 8r + 4 + j: eight units of 8 bytes, each with one 32-bit word per
// half.  Parameters: bf16 [n_kv][max_pos][2][2], (s, m) per half.
#include <cmath>
#include <cstdio>

#include "kernels.h"
#include "tts_decode.h"

namespace tts {
namespace {

constexpr int kRowBytes = 64;
constexpr int kMaxSplitUnits = 160;  // split partials per kv head x kv heads, about one per SM
constexpr int kKv4MaxPos = 1 << 20;
constexpr int kKv4MaxHeads = 4096;

struct RopeRow {
    double c[kHeadDim / 2], s[kHeadDim / 2];
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
        const T c = (T)rope.c[i], s = (T)rope.s[i];
        o[j] = lane < 16 ? a[j] * c - partner * s : a[j] * c + partner * s;
    }
}

// One block per kv head; its warps share the positions, each keeping a
// running maximum, sum and output per query head.
template <int G>
__global__ void __launch_bounds__(256) attn_kv4_kernel(const __grid_constant__ Kv4Params p) {
    __shared__ float wm[8][G], wl[8][G], wo[8][G][kHeadDim];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = blockIdx.x;
    float q[G][4];
#pragma unroll
    for (int j = 0; j < G; ++j) {
        norm_rope<float>(p.qkv + (size_t)(g * G + j) * kHeadDim, p.q_norm, p.rope, p.eps, lane, q[j]);
#pragma unroll
        for (int i = 0; i < 4; ++i) q[j][i] *= 1.0f / sqrtf((float)kHeadDim);
    }
    const size_t base = (size_t)g * p.max_pos;
    if (warp == 0) {
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
    }
    __syncthreads();
    if (warp == 0 && p.kv_row) {
        float x[4];
        const size_t at = base + p.pos;
        load_row(p.k4 + at * kRowBytes, p.k_par + at * 2, lane, x);
        for (int j = 0; j < 4; ++j) p.kv_row[(size_t)g * kHeadDim + 4 * lane + j] = x[j];
        load_row(p.v4 + at * kRowBytes, p.v_par + at * 2, lane, x);
        for (int j = 0; j < 4; ++j) p.kv_row[(size_t)(p.n_kv + g) * kHeadDim + 4 * lane + j] = x[j];
    }
    float m[G], l[G], o[G][4];
#pragma unroll
    for (int j = 0; j < G; ++j) {
        m[j] = -INFINITY;
        l[j] = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) o[j][i] = 0.f;
    }
    for (int t = warp; t <= p.pos; t += 8) {
        float kx[4], vx[4];
        load_row(p.k4 + (base + t) * kRowBytes, p.k_par + (base + t) * 2, lane, kx);
        load_row(p.v4 + (base + t) * kRowBytes, p.v_par + (base + t) * 2, lane, vx);
#pragma unroll
        for (int j = 0; j < G; ++j) {
            const float s = warp_sum(q[j][0] * kx[0] + q[j][1] * kx[1] + q[j][2] * kx[2] + q[j][3] * kx[3]);
            const float mn = fmaxf(m[j], s);
            const float corr = __expf(m[j] - mn), pj = __expf(s - mn);
            l[j] = l[j] * corr + pj;
#pragma unroll
            for (int i = 0; i < 4; ++i) o[j][i] = o[j][i] * corr + pj * vx[i];
            m[j] = mn;
        }
    }
#pragma unroll
    for (int j = 0; j < G; ++j) {
        if (lane == 0) { wm[warp][j] = m[j]; wl[warp][j] = l[j]; }
#pragma unroll
        for (int i = 0; i < 4; ++i) wo[warp][j][4 * lane + i] = o[j][i];
    }
    __syncthreads();
    for (int idx = threadIdx.x; idx < G * kHeadDim; idx += blockDim.x) {
        const int j = idx / kHeadDim, d = idx % kHeadDim;
        float M = wm[0][j];
        for (int w = 1; w < 8; ++w) M = fmaxf(M, wm[w][j]);
        float L = 0.f, O = 0.f;
        for (int w = 0; w < 8; ++w) {
            const float c = wm[w][j] == -INFINITY ? 0.f : __expf(wm[w][j] - M);
            L += wl[w][j] * c;
            O += wo[w][j][d] * c;
        }
        p.out[(size_t)(g * G + j) * kHeadDim + d] = O / L;
    }
}

bool misaligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0; }

int report_kv4(cudaError_t e, const char* what) {
    std::fprintf(stderr, "tts: %s failed: %s\n", what, cudaGetErrorString(e));
    return TTS_ERR_CUDA;
}

int max_splits(int n_kv) { return n_kv >= kMaxSplitUnits ? 1 : kMaxSplitUnits / n_kv; }

// [tickets, one word per kv head][max, sum: 2 words per split and query head]
// [outputs: 128 words per split and query head]
size_t workspace_bytes_for(int n_q, int n_kv) {
    const size_t tickets = ((size_t)n_kv * 4 + 255) & ~(size_t)255;
    return tickets + (size_t)n_q * max_splits(n_kv) * (2 + kHeadDim) * 4;
}

bool heads_ok(int n_q, int n_kv) {
    if (n_kv < 1 || n_q < 1 || n_q > kKv4MaxHeads || n_q % n_kv) return false;
    const int G = n_q / n_kv;
    return G == 1 || G == 2 || G == 4 || G == 8;
}

int rows_ok(const void* k, const void* v, const void* k4, const void* v4, const void* kp, const void* vp, int n_kv,
            int p0, int p1, int stride, int max_pos) {
    if (!k || !v || !k4 || !v4 || !kp || !vp || n_kv < 1 || n_kv > kKv4MaxHeads) return TTS_ERR_ARG;
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
        p.rope.c[i] = std::cos(ang);
        p.rope.s[i] = std::sin(ang);
    }
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    switch (n_q / n_kv) {
        case 1: attn_kv4_kernel<1><<<n_kv, 256, 0, st>>>(p); break;
        case 2: attn_kv4_kernel<2><<<n_kv, 256, 0, st>>>(p); break;
        case 4: attn_kv4_kernel<4><<<n_kv, 256, 0, st>>>(p); break;
        default: attn_kv4_kernel<8><<<n_kv, 256, 0, st>>>(p); break;
    }
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? TTS_OK : report_kv4(e, "tts_attention_decode_kv4");
}
