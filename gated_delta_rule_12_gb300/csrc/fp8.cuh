// fp8.cuh -- values as e4m3 in units of a scale for each block of 128: q = e4m3(y / c), c = max(|y|, 2^-100) / 448 over
// the block, both in fp32 with IEEE rounding.  NaN stays NaN in its place and takes no part in the scale.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"
#include "pairs.cuh"

namespace gdn {

__device__ __forceinline__ float scale_of(float largest) { return fmaxf(largest, kFp8Tiny) / kFp8Max; }

__device__ __forceinline__ float largest(Pair p, float m)
{
    float a, b;
    split(p, a, b);
    return fmaxf(m, fmaxf(fabsf(a), fabsf(b)));
}

// Division by c: the product with its reciprocal, then what is left over once more.  Values next to a border between two
// steps of e4m3 fall where the quotient does; 16-bit inputs lie on such borders often.
struct Unit {
    Pair minus_c, inv;
    // an infinite c takes finite values to 0, infinite ones to NaN
    __device__ __forceinline__ explicit Unit(float c) : minus_c(both(isinf(c) ? 0.f : -c)), inv(both(1.f / c)) {}
    __device__ __forceinline__ Pair operator()(Pair y) const
    {
        const Pair q = mul2(y, inv);
        return fma2(fma2(q, minus_c, y), inv, q);
    }
};

// The first value in the lowest byte; beyond 448 becomes 448.
__device__ __forceinline__ uint32_t pack_e4m3(Pair p, const Unit &unit)
{
    float a, b;
    unsigned short r;
    split(unit(p), a, b);
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
    return r;
}

__device__ __forceinline__ uint32_t pack_e4m3(Pair lo, Pair hi, const Unit &unit)
{
    return pack_e4m3(lo, unit) | pack_e4m3(hi, unit) << 16;
}

}  // namespace gdn
