// Log probabilities of given codes, the entropy of the distribution and its
// top alternatives, from the head's logits (sm_103a).
//
// Bound by reading the logits once (some 6 flops and one exponential a value).
// A warp takes a run of up to 32 NV entries of a row into registers, lane l the
// entries l, l + 32, ..., and finds there the maximum, the sums of e^z and
// z e^z relative to it, and the `top` largest entries, without a second
// reading.  A row of up to 1056 entries is one warp's (four rows a block); a
// longer one is shared by the warps of a block, or by a cluster of blocks when
// there are few rows, whose results are joined through shared memory in a
// fixed order, as a softmax over parts is.
#include <algorithm>
#include <cfloat>
#include <climits>
#include <cmath>
#include <cstdio>

#include <cooperative_groups.h>

#include "fourbit.cuh"
#include "tts_decode.h"

namespace tts {
namespace {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr unsigned kAll = 0xffffffffu;
constexpr int kRunNv = 33;                // 33 values a lane: 1026-entry codebooks in one run
constexpr int kRun = 32 * kRunNv;
// Rows a block, short rows: blocks of 4 leave an SM's registers least idle (4096
// frames x 8 x 1026, 5 alternatives: 29.7 us; 8 rows 30.1, 16 rows 33.5).
constexpr int kShortWarps = 4;
constexpr int kLongWarps = 16;            // warps a block, at most, long rows
// Up to so many alternatives the lanes' maxima are taken one by one to find the
// bound, above it by halving (one by one and by halving, us: 4096 frames x 8 x 1026 with
// 3 alternatives 28.4 and 29.0, 4 28.6 and 29.0, 5 29.6 and 29.7, 6 31.1 and 30.2, 8 32.4
// and 30.8; 40 frames 5 2.9 and 3.0, 8 3.3 and 3.1; 512 x 32000 5 19.7 and 19.8, 6 20.4 and
// 20.3, 16 26.9 and 23.6).
constexpr int kOneByOne = 5;

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float max_nan(float x, float y) {  // NaN where one is
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(y));
    return r;
}
// fp32 bits (no NaN) as unsigned integers in the order of the values; -0 is 0.
__device__ __forceinline__ uint32_t ranked(float z) {
    const uint32_t b = __float_as_uint(z + 0.f);
    return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float from_ranked(uint32_t k) {
    return __uint_as_float((k & 0x80000000u) ? k & 0x7fffffffu : ~k);
}
constexpr uint32_t kRankedNone = 0x007fffffu;  // of -inf

// Differences of logits are taken halved, z / 2 - m / 2, which no pair of finite
// logits overflows, and times c = 2 log2(e) / T they are t = log2(e) (z - m) / T.
__device__ __forceinline__ float halved(float z, float m) { return fmaf(0.5f, z, -0.5f * m); }

// What a part of a row comes to, its NaN entries left out: maximum m, l = sum 2^t, w =
// sum t 2^t, and whether there was a NaN.  l = 0 where nothing is above -inf (and where
// m = +inf, which the caller sees).
struct Part {
    float m, l, w;
    int nan;
};
__device__ __forceinline__ Part join(const Part& a, const Part& b, float c) {
    const float m = fmaxf(a.m, b.m);
    const float ta = halved(a.m, m) * c, tb = halved(b.m, m) * c;
    const float fa = a.l > 0.f ? ex2(ta) : 0.f, fb = b.l > 0.f ? ex2(tb) : 0.f;
    return Part{m, fa * a.l + fb * b.l, (fa > 0.f ? fa * fmaf(ta, a.l, a.w) : 0.f) + (fb > 0.f ? fb * fmaf(tb, b.l, b.w) : 0.f),
                a.nan | b.nan};
}
// All lanes' parts joined, lane order fixed.
__device__ __forceinline__ Part join_lanes(Part a, float c) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const Part b{__shfl_xor_sync(kAll, a.m, o), __shfl_xor_sync(kAll, a.l, o), __shfl_xor_sync(kAll, a.w, o),
                     __shfl_xor_sync(kAll, a.nan, o)};
        a = join(a, b, c);
    }
    return a;
}

// An entry above -inf as one number that orders as the alternatives do: value
// first, then the lower number.
typedef unsigned long long Entry;
__device__ __forceinline__ Entry entry_of(float v, int i) { return (Entry)ranked(v) << 32 | (uint32_t)~i; }
__device__ __forceinline__ float entry_value(Entry e) { return from_ranked((uint32_t)(e >> 32)); }
__device__ __forceinline__ int entry_number(Entry e) { return (int)~(uint32_t)e; }

// Up to 64 candidates for the alternatives, then a sorted list of up to 32 (0: none).
struct Candidates {
    Entry e[64];
};
// The `top` (at most 32) largest of n <= 64 candidates, all different, largest
// first: lane k gets the k-th.  An entry's place is the number of those above it:
// four instructions a candidate, none waiting for another.
__device__ __forceinline__ void sort_candidates(Candidates& c, int n, int top, float& list_v, int& list_i) {
    const int lane = threadIdx.x & 31;
    const Entry a = lane < n ? c.e[lane] : 0, b = lane + 32 < n ? c.e[lane + 32] : 0;
    int place_a = 0, place_b = 0;
    if (n <= 32) {
#pragma unroll 4
        for (int j = 0; j < n; ++j) place_a += c.e[j] > a;
    } else {
#pragma unroll 4
        for (int j = 0; j < n; ++j) {
            const Entry other = c.e[j];
            place_a += other > a;
            place_b += other > b;
        }
    }
    __syncwarp();
    if (a && place_a < top) c.e[place_a] = a;
    if (b && place_b < top) c.e[place_b] = b;
    __syncwarp();
    list_v = -INFINITY;
    if (lane < min(n, top)) {
        list_v = entry_value(c.e[lane]);
        list_i = entry_number(c.e[lane]);
    }
}

// One warp's run z[0 .. n), n <= 32 NV, entries numbered from `first`.  The list
// (list_v, list_i): lane k has the k-th largest entry above -inf found so far
// (-inf: none), equal ones by number; entries of the run join it, all numbered
// above those it came with.
//
// Alternatives: the `top`-th largest of the 32 lanes' maxima is a bound that the
// `top` largest entries reach, and few others do (about 6 for 5, 130 for 32).
// Halving the range between it and the maximum, at most a few times, gives one
// that at least `top` and at most 64 reach; those are gathered and sorted.  Where
// that fails (ties across the bound), with a NaN in the run, or where fewer than
// `top` lanes have an entry above -inf, they are taken out one by one instead.
// (One by one throughout took 41 us on 4096 frames x 8 x 1026 with 5 alternatives
// and 158 us with 32; now 29.5 and 48, and 22 without alternatives.)
template <int NV, bool LISTED>  // LISTED: it comes with a list
__device__ __forceinline__ Part warp_run(const float* z, int n, int first, float c, int top, Candidates& cand,
                                         float& list_v, int& list_i) {
    const int lane = threadIdx.x & 31;
    float v[NV + (NV & 1)];
    if (n >= 32 * (NV - 1)) {  // all but the last load unguarded
#pragma unroll
        for (int i = 0; i < NV - 1; ++i) v[i] = z[lane + 32 * i];
        v[NV - 1] = lane + 32 * (NV - 1) < n ? z[lane + 32 * (NV - 1)] : -INFINITY;
    } else {
#pragma unroll
        for (int i = 0; i < NV; ++i) v[i] = lane + 32 * i < n ? z[lane + 32 * i] : -INFINITY;
    }
    if (NV & 1) v[NV] = -INFINITY;
    // (Loads marked as read once were 2 % faster without alternatives and 12 % slower
    // with 20, which read theirs again.)
    // maxima of chunks of 8 (a NaN is passed over)
    constexpr int kChunks = (NV + 7) / 8;
    float cm[kChunks];
#pragma unroll
    for (int j = 0; j < kChunks; ++j) {
        cm[j] = v[8 * j];
#pragma unroll
        for (int i = 8 * j + 1; i < 8 * j + 8 && i < NV; ++i) cm[j] = fmaxf(cm[j], v[i]);
        cm[j] = fmaxf(cm[j], -INFINITY);
    }
    float m = cm[0];
#pragma unroll
    for (int j = 1; j < kChunks; ++j) m = fmaxf(m, cm[j]);
    Part r;
    r.m = from_ranked(__reduce_max_sync(kAll, ranked(m)));
    r.l = r.w = 0.f;
    if (r.m != -INFINITY && r.m != INFINITY) {
        const f32x2 half = pack2(0.5f, 0.5f), minus = pack2(-0.5f * r.m, -0.5f * r.m), cc = pack2(c, c);
        f32x2 l = pack2(0.f, 0.f), w = l;
#pragma unroll
        for (int i = 0; i < NV; i += 2) {
            // 2^-200 is 0: an entry of -inf adds 0 to w as to l.  A NaN makes both NaN
            const float2 far = unpack2(mul2(fma2(pack2(v[i], v[i + 1]), half, minus), cc));
            const float2 t = make_float2(max_nan(far.x, -200.f), max_nan(far.y, -200.f));
            const f32x2 e = pack2(ex2(t.x), ex2(t.y));
            l = add2(l, e);
            w = fma2(e, pack2(t.x, t.y), w);
        }
        const float2 ls = unpack2(l), wsum = unpack2(w);
        r.l = warp_sum(ls.x + ls.y);
        r.w = warp_sum(wsum.x + wsum.y);
        r.nan = r.l != r.l;
        if (r.nan) r.l = r.w = 0.f;
    } else {
        bool bad = false;
#pragma unroll
        for (int i = 0; i < NV; ++i) bad |= v[i] != v[i];
        r.nan = __any_sync(kAll, bad);
    }
    if (top == 0) return r;

    const float old_v = LISTED ? list_v : -INFINITY;
    const int old_i = list_i;
    // the bound, as a rank
    uint32_t low = 0;
    {
        uint32_t key = ranked(fmaxf(m, old_v));
        if (top <= kOneByOne) {
            for (int k = 0; k < top; ++k) {
                low = __reduce_max_sync(kAll, key);
                if (low <= kRankedNone) break;
                if (lane == __ffs(__ballot_sync(kAll, key == low)) - 1) key = 0;
            }
        } else {  // or a lower one that no more lanes reach, by halving
            uint32_t high = (LISTED ? __reduce_max_sync(kAll, key) : ranked(r.m)) + 1u;
            low = max(__reduce_min_sync(kAll, key), kRankedNone + 1u);
            int reach = __popc(__ballot_sync(kAll, key >= low));
            if (reach < top) low = 0;
            while (reach > top && low + 1u < high) {
                const uint32_t mid = low + (high - low) / 2u;
                const int n = __popc(__ballot_sync(kAll, key >= mid));
                if (n >= top) {
                    low = mid;
                    reach = n;
                } else {
                    high = mid;
                }
            }
        }
    }
    if (low > kRankedNone && !r.nan) {
        constexpr int kWords = (NV + 31) / 32;
        unsigned marks[kWords];
        float bound;
        int count;
        // an entry reaches the bound where (next value below it) - entry is negative:
        // the sign bits, shifted in one by one
        auto mark = [&](uint32_t rank) {
            bound = from_ranked(rank);
            // (the rank below +0 is -0's, which is as large: the one before it)
            const float below = from_ranked(rank == 0x80000000u ? rank - 2 : rank - 1);
            int mine = LISTED && old_v >= bound;
#pragma unroll
            for (int w = 0; w < kWords; ++w) {
                marks[w] = 0;
#pragma unroll
                for (int i = 31; i >= 0; --i)
                    if (32 * w + i < NV) marks[w] = __funnelshift_l(__float_as_uint(below - v[32 * w + i]), marks[w], 1);
                mine += __popc(marks[w]);
            }
            count = __reduce_add_sync(kAll, mine);
        };
        mark(low);
        uint32_t high = ranked(r.m) + 1u;  // reached by none of the run
        if (LISTED) high = max(high, __reduce_max_sync(kAll, ranked(old_v)) + 1u);
        while (count > 64 && low + 1u < high) {
            const uint32_t mid = low + (high - low) / 2u;
            mark(mid);
            if (count >= top) {
                low = mid;
            } else {
                high = mid;
                count = 65;  // not yet
            }
        }
        if (count <= 64) {
            // a lane gives out its marked entries, one a turn: most lanes have none, few
            // have two
            int place = 0;
            auto gather = [&](bool in, float x, int at) {
                const unsigned who = __ballot_sync(kAll, in);
                if (in) cand.e[place + __popc(who & ((1u << lane) - 1))] = entry_of(x, at);
                place += __popc(who);
            };
            if (LISTED) gather(old_v >= bound, old_v, old_i);
#pragma unroll
            for (int w = 0; w < kWords; ++w)
                while (__any_sync(kAll, marks[w] != 0)) {
                    const bool in = marks[w] != 0;
                    const int i = 32 * w + __ffs(marks[w]) - 1;
                    gather(in, in ? z[lane + 32 * i] : 0.f, first + 32 * i + lane);
                    marks[w] &= marks[w] - 1;
                }
            __syncwarp();
            sort_candidates(cand, count, top, list_v, list_i);
            __syncwarp();
            return r;
        }
    }

    float have = old_v;  // the old list's entry while it is not taken: chunk -1, the lowest numbers
    list_v = -INFINITY;
    for (int k = 0; k < top; ++k) {
        float best = have;
#pragma unroll
        for (int j = 0; j < kChunks; ++j) best = fmaxf(best, cm[j]);
        const uint32_t most = __reduce_max_sync(kAll, ranked(best));
        if (most <= kRankedNone) break;
        const float b = from_ranked(most);
        // of the lanes that hold it, the first chunk, then the lowest number in it
        int chunk = kChunks;
#pragma unroll
        for (int j = kChunks - 1; j >= 0; --j)
            if (cm[j] == b) chunk = j;
        if (have == b) chunk = -1;
        chunk = __reduce_min_sync(kAll, chunk);
        int at = INT_MAX;
        if (chunk < 0) {
            if (have == b) at = old_i;
            const int win = __reduce_min_sync(kAll, at);
            if (at == win) have = -INFINITY;
            at = win;
        } else {
#pragma unroll
            for (int j = 0; j < kChunks; ++j)
                if (chunk == j) {
                    int q = -1;
#pragma unroll
                    for (int i = 8 * j + 7; i >= 8 * j; --i)
                        if (i < NV && v[i] == b) q = i;
                    if (q >= 0) at = first + 32 * q + lane;
                    const int win = __reduce_min_sync(kAll, at);
                    if (at != win) q = -1;
                    at = win;
                    cm[j] = -INFINITY;
#pragma unroll
                    for (int i = 8 * j; i < 8 * j + 8 && i < NV; ++i) {
                        if (i == q) v[i] = -INFINITY;
                        cm[j] = fmaxf(cm[j], v[i]);
                    }
                }
        }
        if (lane == k) {
            list_v = b;
            list_i = at;
        }
    }
    return r;
}

// n <= 32 sorted lists merged: lane k gets the k-th entry of all.
__device__ __forceinline__ void merge_lists(const Candidates* lists, int n, int top, float& list_v, int& list_i) {
    const int lane = threadIdx.x & 31;
    int next = 0;
    Entry head = lane < n ? lists[lane].e[0] : 0;
    list_v = -INFINITY;
    for (int k = 0; k < top; ++k) {
        const uint32_t value = (uint32_t)(head >> 32), most = __reduce_max_sync(kAll, value);
        if (most == 0) break;
        const uint32_t win = __reduce_max_sync(kAll, value == most ? (uint32_t)head : 0u);
        if (lane == k) {
            list_v = from_ranked(most);
            list_i = (int)~win;
        }
        if (value == most && (uint32_t)head == win) {
            ++next;
            head = next < 32 ? lists[lane].e[next] : 0;
        }
    }
}

// The results of row-and-codebook `item`, by one warp, from its joined part and
// its list.  A list with fewer than `top` entries above -inf is filled up with
// the -inf entries and then the NaN entries, by number: a search of the row.
__device__ __forceinline__ void finish(const LogprobParams& p, size_t item, const float* z, const Part& r, float list_v,
                                       int list_i) {
    const int lane = threadIdx.x & 31;
    const bool bad = r.nan || r.m == INFINITY, none = !bad && r.m == -INFINITY;
    const float logl = logf(r.l);
    auto logp = [&](float x) { return bad ? NAN : none ? -INFINITY : fmaf(halved(x, r.m), p.two_over_t, -logl); };
    if (lane == 0) {
        if (p.logprob) {
            const int code = p.codes[item];
            p.logprob[item] = code < 0 || code >= p.V ? NAN : logp(z[code]);
        }
        // (the quotient to 2 ulp: as exact as the sums, and 0.2 us less for 4096 frames)
        if (p.entropy) p.entropy[item] = bad ? NAN : none ? 0.f : logl - __fdividef(r.w, r.l) * kLn2;
    }
    if (p.top == 0) return;
    int got = __popc(__ballot_sync(kAll, lane < p.top && list_v != -INFINITY));
    for (int pass = 0; pass < 2 && got < p.top; ++pass)
        for (int i0 = 0; i0 < p.V && got < p.top; i0 += 32) {
            const float x = i0 + lane < p.V ? z[i0 + lane] : 0.f;
            unsigned found = __ballot_sync(kAll, pass ? x != x : x == -INFINITY);
            for (; found && got < p.top; found &= found - 1, ++got)
                if (lane == got) {
                    list_v = -INFINITY;
                    list_i = i0 + __ffs(found) - 1;
                }
        }
    if (lane < p.top) {
        p.top_codes[item * p.top + lane] = list_i;
        p.top_logprob[item * p.top + lane] = logp(list_v);
    }
}

__device__ __forceinline__ const float* row_of(const LogprobParams& p, size_t item) {
    return p.logits + (item / p.n_cb) * p.ld + (item % p.n_cb) * (size_t)p.V;
}

template <int NV>
__global__ void __launch_bounds__(kShortWarps * 32) logprobs_short_kernel(const LogprobParams p, int items) {
    __shared__ Candidates cand[kShortWarps];
    const int item = blockIdx.x * kShortWarps + (threadIdx.x >> 5);
    pdl_trigger();
    pdl_wait();
    if (item >= items) return;
    const float* z = row_of(p, item);
    float list_v = -INFINITY;
    int list_i = 0;
    const Part r = warp_run<NV, false>(z, p.V, 0, kLog2e * p.two_over_t, p.top, cand[threadIdx.x >> 5], list_v, list_i);
    finish(p, item, z, r, list_v, list_i);
}

// A cluster of gridDim.y blocks a row: its warps take runs of the row in turn.
__global__ void __launch_bounds__(kLongWarps * 32, 2) logprobs_long_kernel(const LogprobParams p) {
    __shared__ Part parts[kLongWarps];
    // a warp's gathered entries, then its list; and in a cluster the blocks' lists,
    // which they hand to the first
    extern __shared__ Candidates lists[];
    __shared__ Part block_part[8];
    namespace cg = cooperative_groups;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, W = blockDim.x >> 5, C = gridDim.y;
    Candidates* block_list = lists + W;
    if (C > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");  // all blocks run: awaited below
    pdl_trigger();
    pdl_wait();
    const size_t item = blockIdx.x;
    const float* z = row_of(p, item);
    const float c = kLog2e * p.two_over_t;
    Part r{-INFINITY, 0.f, 0.f, 0};
    float list_v = -INFINITY;
    int list_i = 0;
    for (int first = ((int)blockIdx.y * W + warp) * kRun; first < p.V; first += C * W * kRun)
        r = join(r, warp_run<kRunNv, true>(z + first, min(kRun, p.V - first), first, c, p.top, lists[warp], list_v, list_i), c);
    if (lane == 0) parts[warp] = r;
    lists[warp].e[lane] = list_v == -INFINITY ? 0 : entry_of(list_v, list_i);
    if (C > 1) asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
    __syncthreads();
    if (warp == 0) {
        r = join_lanes(lane < W ? parts[lane] : Part{-INFINITY, 0.f, 0.f, 0}, c);
        merge_lists(lists, W, p.top, list_v, list_i);
        if (C == 1) {
            finish(p, item, z, r, list_v, list_i);
        } else {
            const auto cluster = cg::this_cluster();
            const unsigned at = blockIdx.y;
            if (lane == 0) *cluster.map_shared_rank(&block_part[at], 0) = r;
            *cluster.map_shared_rank(&block_list[at].e[lane], 0) = list_v == -INFINITY ? 0 : entry_of(list_v, list_i);
        }
    }
    if (C == 1) return;
    cg::this_cluster().sync();
    if (blockIdx.y != 0 || warp != 0) return;
    r = join_lanes(lane < C ? block_part[lane] : Part{-INFINITY, 0.f, 0.f, 0}, c);
    merge_lists(block_list, C, p.top, list_v, list_i);
    finish(p, item, z, r, list_v, list_i);
}

// How a long row is shared: warps a block, blocks a row.
struct LongPlan {
    int warps, blocks;
};
LongPlan plan_long(int items, int V, int sms) {
    // Warps a row, each with its runs in turn: the least rounds of blocks (32 warps
    // an SM) times turns, and of equals the fewest, four at least, as there are fewer
    // lists to merge and few entries of a later run are above a warp's list.  (20
    // alternatives: 512 x 32000 8 warps 25.3 us, 11 warps 30.4, 16 warps 28.6;
    // 2000 x 8192 4 warps 26.4, 2 warps 27.8, 8 warps 32.9.)
    const int runs = (V + kRun - 1) / kRun;
    int W = std::min(kLongWarps, runs);
    const auto cost = [&](int w) {
        const long long at_once = (long long)sms * (32 / w);
        return (items + at_once - 1) / at_once * ((runs + w - 1) / w);
    };
    for (int w = W - 1; w >= 4; --w)
        if (cost(w) <= cost(W)) W = w;
    // one block a row, or so many that every warp has one run, while the rows do
    // not fill the SMs by themselves
    int C = 1;
    while (C < 8 && C * W < runs && (long long)items * C < sms) C *= 2;
    return LongPlan{W, C};
}

}  // namespace

cudaError_t launch_logprobs(const LogprobParams& p, cudaStream_t s) {
    const int items = p.rows * p.n_cb;  // below 2^31: checked by the caller
    if (p.V <= kRun) {
        const unsigned grid = (items + kShortWarps - 1) / kShortWarps;
        // 8 values a lane where that is enough: the 33 of a longer run would be
        // mostly padding
        return launch_ordered(p.V <= 256 ? logprobs_short_kernel<8> : logprobs_short_kernel<kRunNv>, dim3(grid),
                              dim3(kShortWarps * 32), 0, s, 1, 1, p, items);
    }
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    const LongPlan plan = plan_long(items, p.V, sms);
    const int W = plan.warps, C = plan.blocks;
    const size_t smem = sizeof(Candidates) * (W + (C > 1 ? C : 0));
    return launch_ordered(logprobs_long_kernel, dim3(items, C), dim3(W * 32), smem, s, C, 1, p);
}

}  // namespace tts

extern "C" int tts_code_logprobs(const float* logits, long long ld, const int32_t* codes, int rows, int n_cb,
                                 int cb_vocab, float temperature, int top, float* logprob, float* entropy,
                                 int32_t* top_codes, float* top_logprob, void* stream) {
    using namespace tts;
    if (rows < 0 || n_cb < 1 || n_cb > kMaxCodebooks || cb_vocab < 2 || cb_vocab > (1 << 20)) return TTS_ERR_ARG;
    if (ld < (long long)n_cb * cb_vocab || top < 0 || top > kMaxTop || top > cb_vocab) return TTS_ERR_ARG;
    if ((long long)rows * n_cb > 0x7fffffffLL - kShortWarps) return TTS_ERR_ARG;
    if (!(temperature >= FLT_MIN) || !std::isfinite(temperature)) return TTS_ERR_ARG;
    if (rows == 0) return TTS_OK;  // an empty array may have no address
    if (!logits || (logprob != nullptr) != (codes != nullptr)) return TTS_ERR_ARG;
    if ((top > 0) != (top_codes != nullptr) || (top > 0) != (top_logprob != nullptr)) return TTS_ERR_ARG;
    const uintptr_t all = reinterpret_cast<uintptr_t>(logits) | reinterpret_cast<uintptr_t>(codes) |
                          reinterpret_cast<uintptr_t>(logprob) | reinterpret_cast<uintptr_t>(entropy) |
                          reinterpret_cast<uintptr_t>(top_codes) | reinterpret_cast<uintptr_t>(top_logprob);
    if (all & 3) return TTS_ERR_ARG;
    if (rows > 1 && ld > (1LL << 48) / rows) return TTS_ERR_ARG;  // no memory is that large
    const size_t n = (size_t)rows * n_cb, row = (size_t)n_cb * cb_vocab;
    if (overwritten({{logprob, 4 * n}, {entropy, 4 * n}, {top_codes, 4 * n * top}, {top_logprob, 4 * n * top}},
                    {{logits, 4 * ((size_t)(rows - 1) * ld + row)}, {codes, 4 * n}}))
        return TTS_ERR_ARG;
    LogprobParams p{logits, ld, codes, rows, n_cb, cb_vocab, 2.f / temperature, top, logprob, entropy, top_codes,
                    top_logprob};
    const cudaError_t e = launch_logprobs(p, static_cast<cudaStream_t>(stream));
    if (e == cudaSuccess) return TTS_OK;
    std::fprintf(stderr, "tts: tts_code_logprobs failed: %s\n", cudaGetErrorString(e));
    return TTS_ERR_CUDA;
}
