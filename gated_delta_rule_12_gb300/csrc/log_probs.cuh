// log_probs.cuh -- what the log probabilities of given tokens take beyond the cross entropy, on the tensor cores and on the
// CUDA cores alike: a row's statistics over a part of the vocabulary, its best words in order, and how parts join.
//
//     lse = T + log S,  H = lse - sum_v p_v l_v = log S - U / S,   T = max l_v,  S = sum e^(l_v - T),  U = sum e^(l_v - T) (l_v - T)
// U and log S have no large terms that cancel: H is the sum of two positive numbers.  Moving T moves U by (old - new) S.
//
// Words are ordered by their logit, equal ones by the lower index.  A logit of -inf or NaN is no alternative.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "kernels.h"
#include "part_order.h"

namespace gdn {

constexpr int kMostTop = 20;

// A part's statistics; the words among its best that may be among the row's.
struct RowStat {
    float top, sum, u;    // top: 0 in place of +inf, which stays in the sum
    int count;
};

// The K best words so far, best first.  Words come with rising indexes.
template <int K>
struct BestWords {
    float v[K];
    int id[K];
    __device__ __forceinline__ BestWords()
    {
#pragma unroll
        for (int i = 0; i < K; ++i) {
            v[i] = -INFINITY;
            id[i] = -1;
        }
    }
    __device__ __forceinline__ void add(float x, int word)   // nothing changes unless x is above the last
    {
#pragma unroll
        for (int i = K - 1; i > 0; --i) {
            const bool over = x > v[i - 1], here = x > v[i];
            id[i] = over ? id[i - 1] : here ? word : id[i];
            v[i] = over ? v[i - 1] : here ? x : v[i];
        }
        id[0] = x > v[0] ? word : id[0];
        v[0] = x > v[0] ? x : v[0];
    }
    __device__ __forceinline__ void pop()
    {
#pragma unroll
        for (int i = 0; i + 1 < K; ++i) {
            v[i] = v[i + 1];
            id[i] = id[i + 1];
        }
        v[K - 1] = -INFINITY;
        id[K - 1] = -1;
    }
    __device__ __forceinline__ float value(int n) const   // of the word in place n
    {
        float x = v[0];
#pragma unroll
        for (int i = 1; i < K; ++i) x = i == n ? v[i] : x;
        return x;
    }
    __device__ __forceinline__ int count(int most) const
    {
        int n = 0;
#pragma unroll
        for (int i = 0; i < K; ++i) n += i < most && id[i] >= 0;
        return n;
    }
};

// Floats as whole numbers of the same order, both zeros as one; 0 is below all of them.
__device__ __forceinline__ unsigned order_of(float x)
{
    const unsigned b = __float_as_uint(x + 0.f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// The largest float below the one of this place.
__device__ __forceinline__ float below(unsigned place)
{
    const unsigned p = place == 0x80000000u ? 0x7ffffffeu : place - 1u;   // below zero comes the least negative number
    return __uint_as_float(p & 0x80000000u ? p & 0x7fffffffu : ~p);
}

// Sorts 32 values, largest first: a bitonic network, 240 exchanges.  (By recursion, as loops whose steps double are not
// unrolled and would leave the values in memory.)
template <int RUN = 2, int APART = 1>
__device__ __forceinline__ void sort32(float (&v)[32])
{
#pragma unroll
    for (int i = 0; i < 32; ++i)
        if (!(i & APART)) {
            const float a = v[i], b = v[i + APART], high = fmaxf(a, b), low = fminf(a, b);
            v[i] = i & RUN ? low : high;
            v[i + APART] = i & RUN ? high : low;
        }
    if constexpr (APART > 1) sort32<RUN, APART / 2>(v);
    else if constexpr (RUN < 32) sort32<RUN * 2, RUN>(v);
}

// A warp's lists to the row's k best words.
template <int K>
__device__ __forceinline__ void write_best(BestWords<K> &best, int k, float lse, bool keep, int *ids, float *logps)
{
    const int lane = threadIdx.x & 31;
    for (int i = 0; i < k; ++i) {
        const unsigned mine = best.id[0] >= 0 ? order_of(best.v[0]) : 0u;
        const unsigned high = __reduce_max_sync(0xffffffffu, mine);
        const unsigned word = __reduce_min_sync(0xffffffffu, high && mine == high ? (unsigned)best.id[0] : 0xffffffffu);
        if (high && mine == high && (unsigned)best.id[0] == word) {
            ids[i] = keep ? best.id[0] : -1;
            logps[i] = keep ? best.v[0] - lse : 0.f;
            best.pop();
        }
        if (!high && lane == 0) {   // fewer words than asked for
            ids[i] = -1;
            logps[i] = keep ? -INFINITY : 0.f;
        }
    }
}

// The parts of the rows, and of each its best words, `top` of them.
struct LogProbParts {
    const RowStat *stat;
    const float2 *best;       // a logit and its word's bits, best first
    const float *at;          // [N] the targets' logits
    const int32_t *targets;
    const unsigned *cut;      // [N] order_of() of a logit that the row's best words do not fall below (0: none); or null
    int N, V, top;
    int parts;                // [N][parts] where order.pairs = 0: every row has all of them
    PartOrder order;          // else as this has them
};

// Joins a row's parts, a warp a row, in a fixed order; K: the best words that a lane keeps, at least p.top.
template <int K>
static __global__ void __launch_bounds__(256) logp_join_kernel(LogProbParts p, LogProbs out)
{
    const int lane = threadIdx.x & 31;
    const int64_t row = ((int64_t)blockIdx.x * 256 + threadIdx.x) >> 5;
    asm volatile("griddepcontrol.wait;" ::: "memory");   // launched beside the kernel that writes the parts
    if (row >= p.N) return;
    const bool ordered = p.order.pairs > 0;
    const int row_tile = (int)(row / PartOrder::kRows), parts = ordered ? p.order.of(row_tile).parts : p.parts;
    const int64_t start = ordered ? p.order.first((int)row) : row * p.parts, step = ordered ? p.order.step((int)row, p.N) : 1;
    const RowStat *stat = p.stat + start;
    const unsigned told = K && p.cut ? p.cut[row] : 0u;
    const float cut = told ? below(told) : -INFINITY;   // the row's best words are above it
    float top = -INFINITY, sum = 0.f, u = 0.f;
    // Moves (sum, u) from `top` to a higher reference and adds another's.  A part without words has -inf and zeros (or NaN).
    auto join = [&](float t, float s, float v) {
        const float to = fmaxf(top, t), base = to == -INFINITY ? 0.f : to;
        const float da = fmaxf(top - base, -1e4f), db = fmaxf(t - base, -1e4f), fa = expf(da), fb = expf(db);
        u = fa * fmaf(da, sum, u) + fb * fmaf(db, s, v);
        sum = fmaf(fa, sum, fb * s);
        top = to;
    };
    BestWords<K ? K : 1> best;
    for (int first = lane; first < parts; first += 128) {   // four parts at a time, on their way together
        float4 v[4];
        bool in[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int i = first + 32 * j;
            in[j] = i < parts && (!ordered || p.order.has(row_tile, i));
            v[j] = in[j] ? *reinterpret_cast<const float4 *>(stat + i * step) : make_float4(-INFINITY, 0.f, 0.f, 0.f);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (!in[j]) continue;
            join(v[j].x, v[j].y, v[j].z);
            if (K && !(v[j].x < cut && v[j].y < INFINITY)) {   // (an infinite maximum, 0 here, leaves an infinite sum)
                const int count = __float_as_int(v[j].w);
                const float2 *words = p.best + (start + (first + 32 * j) * step) * p.top;
                for (int c = 0; c < count; c += 4) {
                    float2 w[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) w[e] = c + e < count ? words[c + e] : make_float2(-INFINITY, 0.f);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (w[e].x > cut && w[e].x > best.v[K ? K - 1 : 0]) best.add(w[e].x, __float_as_int(w[e].y));
                    if (!(w[3].x > cut)) break;   // nor are the worse ones
                }
            }
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        join(__shfl_xor_sync(0xffffffffu, top, o), __shfl_xor_sync(0xffffffffu, sum, o), __shfl_xor_sync(0xffffffffu, u, o));
    const float base = top == -INFINITY ? 0.f : top;
    const int t = p.targets[row];
    const bool keep = t >= 0 && t < p.V;
    const float ls = logf(sum), lse = base + ls;
    if (lane == 0) {
        out.logp[row] = keep ? (p.at[row] - base) - ls : 0.f;
        out.entropy[row] = keep ? ls - u / sum : 0.f;
        if (out.lse) out.lse[row] = keep ? lse : 0.f;
    }
    if (K) write_best(best, p.top, lse, keep, out.top_ids + row * p.top, out.top_logps + row * p.top);
}

}  // namespace gdn
