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

// The parts of the rows, part n of row r at n * part_step + r * row_step, and its best words, `top` of them, likewise.
struct LogProbParts {
    const RowStat *stat;
    const float2 *best;       // a logit and its word's bits, best first
    const float *at;          // [N] the targets' logits
    const int32_t *targets;
    int64_t part_step, row_step;
    int N, V, parts, top;
};

// Joins a row's parts, a warp a row, in a fixed order; K: the best words that a lane keeps, at least p.top.
template <int K>
static __global__ void __launch_bounds__(256) logp_join_kernel(LogProbParts p, LogProbs out)
{
    const int lane = threadIdx.x & 31;
    const int64_t row = ((int64_t)blockIdx.x * 256 + threadIdx.x) >> 5;
    asm volatile("griddepcontrol.wait;" ::: "memory");   // launched beside the kernel that writes the parts
    if (row >= p.N) return;
    const RowStat *stat = p.stat + row * p.row_step;
    float top = -INFINITY;
#pragma unroll 4
    for (int i = lane; i < p.parts; i += 32) top = fmaxf(top, stat[i * p.part_step].top);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    const float base = isinf(top) ? 0.f : top;   // keeps infinities and NaN in the sum
    float sum = 0.f, u = 0.f;
    BestWords<K ? K : 1> best;
    for (int i = lane; i < p.parts; i += 32) {
        const float4 v = *reinterpret_cast<const float4 *>(stat + i * p.part_step);
        const float d = v.x - base, f = expf(d);
        sum = fmaf(v.y, f, sum);
        u = fmaf(f, fmaf(v.x == -INFINITY ? 0.f : d, v.y, v.z), u);
        if (K) {
            const int count = __float_as_int(v.w);
            const float2 *words = p.best + (i * p.part_step + row * p.row_step) * p.top;
            for (int c = 0; c < count; c += 4) {   // a few at a time, on their way together
                float2 w[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) w[j] = c + j < count ? words[c + j] : make_float2(-INFINITY, 0.f);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (w[j].x > best.v[K ? K - 1 : 0]) best.add(w[j].x, __float_as_int(w[j].y));
            }
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        sum += __shfl_xor_sync(0xffffffffu, sum, o);
        u += __shfl_xor_sync(0xffffffffu, u, o);
    }
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
