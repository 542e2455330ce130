// rows.cuh -- what the norms' kernels share: a team of threads holds a row in registers, rows come ahead through
// asynchronous copies into shared memory, and sums over a row go over the team.
#pragma once

#include "common.cuh"
#include "pairs.cuh"

namespace gdn {
namespace rows {

constexpr int kSMs = 152;
static_assert(kSMs % 8 == 0, "a team's rows all have to start at the same place of a 16-byte chunk");

// VW elements as one access: 16 bytes, or two bf16 or one element where rows are not aligned for more.
template <typename T, int VW>
struct Raw {
    static constexpr int kWords = VW * sizeof(T) / 4 > 0 ? VW * sizeof(T) / 4 : 1;
    uint32_t w[kWords];
    __device__ __forceinline__ float get(int j) const
    {
        if constexpr (sizeof(T) == 4) return __uint_as_float(w[j]);
        else return __uint_as_float(j & 1 ? w[j / 2] & 0xffff0000u : w[j / 2] << 16);
    }
    __device__ __forceinline__ void drop(int n)   // the first n elements become 0
    {
#pragma unroll
        for (int k = 0; k < kWords; ++k)
            if constexpr (sizeof(T) == 4) w[k] = k < n ? 0u : w[k];
            else w[k] = 2 * k + 1 < n ? 0u : 2 * k < n ? w[k] & 0xffff0000u : w[k];
    }
};

// Rows on their way: every thread copies its own accesses into its own slots, kStages rows ahead, and reads them back
// itself, so the ring needs no barrier and no registers.  A missing access reads as zeros.  Single bf16 elements have
// no asynchronous copy and go through a register.  MAX threads' slots take up to 128 KB.
template <typename T, int VW, int NV, int TENSORS, int MAX>
struct Ring {
    static constexpr int kBytes = Raw<T, VW>::kWords * 4;
    static constexpr int kFit = 128 * 1024 / (TENSORS * NV * kBytes * (MAX < 512 ? 512 : MAX));
    static constexpr int kStages = kFit >= 4 ? 4 : kFit >= 2 ? 2 : 1;
    uint32_t base;
    static __host__ __device__ int stage_bytes(int threads) { return TENSORS * NV * kBytes * threads; }
    static __host__ __device__ int bytes(int threads) { return kStages * stage_bytes(threads); }
    __device__ __forceinline__ explicit Ring(const void *smem)
        : base(static_cast<uint32_t>(__cvta_generic_to_shared(smem)) + threadIdx.x * kBytes) {}
    __device__ __forceinline__ uint32_t slot(int stage, int tensor, int v) const
    {
        return base + ((stage * TENSORS + tensor) * NV + v) * (blockDim.x * kBytes);
    }
    __device__ __forceinline__ void load(int stage, int tensor, int v, const T *p, bool in) const   // p is read if `in`
    {
        if constexpr (kBytes == 16)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;"
                         :: "r"(slot(stage, tensor, v)), "l"(p), "r"(in ? 16 : 0) : "memory");
        else if constexpr (VW * sizeof(T) == 4)
            asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;"
                         :: "r"(slot(stage, tensor, v)), "l"(p), "r"(in ? 4 : 0) : "memory");
        else
            asm volatile("st.shared.b32 [%0], %1;"
                         :: "r"(slot(stage, tensor, v)),
                            "r"(in ? (uint32_t)__ldcs(reinterpret_cast<const unsigned short *>(p)) : 0u) : "memory");
    }
    // the first `left` elements of an access of 16 bytes, zeros behind them
    __device__ __forceinline__ void load_some(int stage, int tensor, int v, const T *p, int left) const
    {
        const int bytes = min(max(left * (int)sizeof(T), 0), 16);
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;"
                     :: "r"(slot(stage, tensor, v)), "l"(p), "r"(bytes) : "memory");
    }
    template <int N>
    __device__ __forceinline__ void read(int stage, int tensor, Raw<T, VW> (&r)[N], int from = 0) const
    {
#pragma unroll
        for (int v = 0; v < N; ++v)
            if constexpr (kBytes == 16)
                asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                             : "=r"(r[v].w[0]), "=r"(r[v].w[1]), "=r"(r[v].w[2]), "=r"(r[v].w[3])
                             : "r"(slot(stage, tensor, from + v)) : "memory");
            else
                asm volatile("ld.shared.b32 %0, [%1];"
                             : "=r"(r[v].w[0]) : "r"(slot(stage, tensor, from + v)) : "memory");
    }
};

__device__ __forceinline__ void commit_copies() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void wait_copies() { asm volatile("cp.async.wait_group %0;" :: "n"(N) : "memory"); }

// A thread's NV accesses as pairs: pair i holds elements 2 i and 2 i + 1 of the NV * VW.
template <typename T, int VW, int NV>
__device__ __forceinline__ Pair get_pair(const Raw<T, VW> (&raw)[NV], int i)
{
    if constexpr (VW == 1) return pair(raw[2 * i].get(0), raw[2 * i + 1].get(0));
    else return pair(raw[2 * i / VW].get(2 * i % VW), raw[2 * i / VW].get(2 * i % VW + 1));
}

// Access v of the row at `row`, at column c.
template <typename T, int VW, int N>
__device__ __forceinline__ void put(T *p, const Pair (&y)[N], int v)
{
    if constexpr (VW == 1) {
        float a, b;
        split(y[v / 2], a, b);
        *p = from_f32<T>(v & 1 ? b : a);
    } else if constexpr (VW == 2) {
        float a, b;
        uint32_t w;
        split(y[v], a, b);
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(b), "f"(a));
        *reinterpret_cast<uint32_t *>(p) = w;
    } else if constexpr (sizeof(T) == 4) {
        float4 r;
        split(y[2 * v], r.x, r.y);
        split(y[2 * v + 1], r.z, r.w);
        *reinterpret_cast<float4 *>(p) = r;
    } else {
        uint4 r;
        uint32_t *w = reinterpret_cast<uint32_t *>(&r);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float a, b;
            split(y[4 * v + i], a, b);
            asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(b), "f"(a));
        }
        *reinterpret_cast<uint4 *>(p) = r;
    }
}

// The same for an access of which only columns c to c + VW - 1 within [0, D) are the row's.
template <typename T, int VW, int N>
__device__ __forceinline__ void put_some(T *p, const Pair (&y)[N], int v, int c, int D)
{
#pragma unroll
    for (int j = 0; j < VW; ++j) {
        float e[2];
        split(y[(v * VW + j) / 2], e[0], e[1]);
        if (c + j >= 0 && c + j < D) p[j] = from_f32<T>(e[j & 1]);
    }
}

__device__ __forceinline__ float total(Pair p)
{
    float a, b;
    split(p, a, b);
    return a + b;
}

// Sums of N values over a team, the same bits in every thread of it: shuffles within a warp, then, for teams of
// several warps, their sums in order through `sh` behind a barrier of the team's own.
template <int TEAM, int N>
struct TeamSum {
    float *mine, *all;   // where the warp's sums go, where the team's start
    int size, barrier, other;
    __device__ __forceinline__ TeamSum(float *sh, int team_size)   // sh: [2][N][32], a team's part in whole float4s
    {
        size = team_size;
        const int team = threadIdx.x / team_size;
        barrier = 1 + team;
        all = sh + team * ((team_size + 127) / 128 * 4);
        mine = all + threadIdx.x % team_size / 32;
        other = N * 32;      // by turns, so that one barrier a sum is enough
        if constexpr (TEAM == 0) {
            for (int i = threadIdx.x; i < 2 * N * 32; i += blockDim.x) sh[i] = 0.f;
            __syncthreads();
        }
    }
    __device__ __forceinline__ void operator()(float (&v)[N])
    {
#pragma unroll
        for (int o = (TEAM ? TEAM : 32) / 2; o > 0; o >>= 1)
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
        if constexpr (TEAM == 0) {
            if ((threadIdx.x & 31) == 0)
#pragma unroll
                for (int i = 0; i < N; ++i) mine[i * 32] = v[i];
            asm volatile("bar.sync %0, %1;" :: "r"(barrier), "r"(size) : "memory");
            if (size == 64) {
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    const float2 p = *reinterpret_cast<const float2 *>(all + i * 32);
                    v[i] = p.x + p.y;
                }
            } else {
#pragma unroll
                for (int i = 0; i < N; ++i) v[i] = 0.f;
#pragma unroll 1   // unrolled, it makes the backward kernels spill (8192 x 2048 bf16 28 us)
                for (int w = 0; 32 * w < size; w += 4)
#pragma unroll
                    for (int i = 0; i < N; ++i) {
                        const float4 p = *reinterpret_cast<const float4 *>(all + i * 32 + w);
                        v[i] += (p.x + p.y) + (p.z + p.w);
                    }
            }
            mine += other;
            all += other;
            other = -other;
        }
    }
};

// 1 / sqrt(v): the hardware's approximation and one step of Newton's iteration (1 ulp; the division and square root
// of IEEE rounding take 30 instructions a row more).
__device__ __forceinline__ float inv_sqrt(float v)
{
    const float r = rsqrtf(v);
    const float e = fmaf(v * r, -r, 1.f);
    return r > 0.f && r < 1e18f ? fmaf(0.5f * r, e, r) : r;   // v = 0 and infinite v have no step
}

// How rows lie to the accesses.
//   kPartial  every row starts with an access, the last may be missing for some threads.
//   kFull     the same, and the row fills the team: no access is missing.
//   kShifted  rows of any length in tensors that start on 16-byte boundaries: the accesses are the 16-byte chunks of
//             memory, and the first and the last of a row hold elements of its neighbours.  The grid's teams are a
//             multiple of 8, so a team's rows all start at the same place of their first chunk (`ph` elements into it)
//             and its threads keep their columns.
enum { kPartial, kFull, kShifted };

// Stages of the backward kernel's ring for teams of more than 512 threads, 16 elements each: what fits beside the weight.
__host__ __device__ constexpr int again_stages(int stage_bytes, int threads)
{
    return 2 * stage_bytes + 64 * threads <= 226 * 1024 ? 2 : 1;
}

constexpr int kMost = 16384;   // elements of a row that 1024 threads hold

struct Shape { int team, wide; };   // threads a row; 0: `few` accesses each, 1: `many`, 2: three quarters of many

// The smallest team, whole warps up to 1024 threads, that can take the row at `many` accesses a thread; a part of a
// warp, or a warp, at `few` where that is enough.  (Powers of two alone: 8192 x 2049 bf16 35 us forward, 39.6
// backward; whole warps 28 and 29.8.)  8192 x 2048 bf16: forward 32 elements a thread 14.8 us, 16
// elements 15.5, 8 elements 19.8; backward, whose dw and db take twice as many registers, 16 elements 25.2 us,
// 8 elements 29.4, 32 elements (spilling) 51.
inline Shape shape(int D, int vw, int few, int many)
{
    const int nvec = ceil_div(D, vw);
    for (int g = 8; g <= 32; g *= 2)
        if (nvec <= g * few) return {g, 0};
    return {ceil_div(ceil_div(nvec, many), 32) * 32, 1};
}

}  // namespace rows
}  // namespace gdn
