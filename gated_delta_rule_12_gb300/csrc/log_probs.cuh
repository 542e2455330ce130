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

// A warp's lists to the row's k best words.
template <int K>
__device__ __forceinline__ void write_best(BestWords<K> &best, int k, float lse, bool keep, int *ids, float *logps)
{
    const int lane = threadIdx.x & 31;
    for (int i = 0; i < k; ++i) {
        const unsigned mine = best.id[0] >= 0 ? order_of(best.v[0]) : 0u;
        const unsigned high = __reduce_max_sync(0xffffffffu, mine);
        const unsigned word = __reduce_min_sync(0xffffffffu, high && mine == high ? (unsigned)best.id[0] : 0xffffffffu);
        const bool won = high && mine == high && (unsigned)best.id[0] == word;
        if (won) {
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

}  // namespace gdn
