// fp8_quant.cu -- values to e4m3 with a scale for each block of 128 columns of a row (activations), or of 128 rows by 128
// columns (weights):  c = max(|x|, 2^-100) / 448 over the block,  q = e4m3(x / c).
//
// Bound by memory: x read once, q and the scales written.  A block of a row lies in the registers of the 16 (bf16) or 32
// (fp32) threads that read it in 16-byte accesses, its maximum goes by shuffles; a 128 x 128 block in those of a CTA.
// Rows that 16-byte accesses do not fit go element by element.
//
// Measured (GB300, device time): 8192 x 2048 bf16 10.2 us, 5.0 TB/s (four blocks of a thread on their way instead of two 11.8,
// eight 12.5 to 13.1; a CTA for each two instead of a grid that stays 10.5); fp32 17.1 us, 4.9 TB/s.  Weights of 6144 x 2048, a
// CTA a block: bf16 12.8 us, 3.0 TB/s, fp32 12.4, 5.1.
#include "common.cuh"
#include "fp8.cuh"
#include "kernels.h"

namespace gdn {
namespace {

constexpr int kThreads = 256;

template <typename T>
struct Chunk {      // 16 bytes
    static constexpr int kSize = 16 / sizeof(T);
    uint4 v;
    __device__ __forceinline__ Pair get(int i) const   // elements 2 i and 2 i + 1
    {
        const uint32_t *w = reinterpret_cast<const uint32_t *>(&v);
        if constexpr (sizeof(T) == 4) return pair(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
        else return pair(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
    }
    __device__ __forceinline__ float most() const
    {
        float m = 0.f;
#pragma unroll
        for (int i = 0; i < kSize / 2; ++i) m = largest(get(i), m);
        return m;
    }
    __device__ __forceinline__ void put(unsigned char *to, const Unit &unit) const
    {
        if constexpr (kSize == 8)
            *reinterpret_cast<uint2 *>(to) = make_uint2(pack_e4m3(get(0), get(1), unit), pack_e4m3(get(2), get(3), unit));
        else
            *reinterpret_cast<uint32_t *>(to) = pack_e4m3(get(0), get(1), unit);
    }
};

// Blocks of a row.  EVEN: rows are whole blocks, so block i of all starts at element 128 i.
template <typename T, bool EVEN>
__global__ void __launch_bounds__(kThreads) rows_kernel(const Fp8QuantArgs a, int64_t items, unsigned per_row)
{
    constexpr int VW = Chunk<T>::kSize, kLanes = kFp8Block / VW, kAhead = 2;
    const int lane = threadIdx.x % kLanes;
    const int64_t step = (int64_t)gridDim.x * (kThreads / kLanes);
    // the threads of a warp stay together: a block behind the last reads as zeros
    for (int64_t first = (int64_t)blockIdx.x * (kThreads / kLanes); first < items; first += kAhead * step) {
        Chunk<T> x[kAhead];
        int64_t at[kAhead], item[kAhead];
        bool in[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            item[k] = first + k * step + threadIdx.x / kLanes;
            in[k] = item[k] < items;
            if constexpr (EVEN) {
                at[k] = item[k] * kFp8Block + lane * VW;
            } else {
                const int64_t row = items < (int64_t)1 << 32 ? (int64_t)((unsigned)item[k] / per_row) : item[k] / per_row;
                const int64_t col = (item[k] - row * per_row) * kFp8Block + lane * VW;
                at[k] = row * a.D + col;
                in[k] = in[k] && col < a.D;
            }
            x[k].v = in[k] ? __ldcs(reinterpret_cast<const uint4 *>((const T *)a.x + at[k])) : make_uint4(0u, 0u, 0u, 0u);
        }
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            float m = x[k].most();
#pragma unroll
            for (int o = kLanes / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
            const float c = scale_of(m);
            if (in[k]) {
                x[k].put(a.q + at[k], Unit(c));
                if (lane == 0) a.scales[item[k]] = c;
            }
        }
    }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) rows_any_kernel(const Fp8QuantArgs a, int64_t items, unsigned per_row)
{
    const int lane = threadIdx.x & 31;
    for (int64_t i = (int64_t)blockIdx.x * (kThreads / 32) + threadIdx.x / 32; i < items;
         i += (int64_t)gridDim.x * (kThreads / 32)) {
        const int64_t row = i / per_row, col = (i - row * per_row) * kFp8Block + lane;
        float x[4], m = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            x[j] = col + 32 * j < a.D ? to_f32(((const T *)a.x)[row * a.D + col + 32 * j]) : 0.f;
            m = fmaxf(m, fabsf(x[j]));
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        const float c = scale_of(m);
        const Unit unit(c);
        if (lane == 0) a.scales[i] = c;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (col + 32 * j < a.D) a.q[row * a.D + col + 32 * j] = (unsigned char)pack_e4m3(both(x[j]), unit);
    }
}

__device__ __forceinline__ float block_max(float m)
{
    __shared__ float sh[kThreads / 32];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) m = fmaxf(m, sh[i]);
    return m;
}

// 128 x 128 blocks, one a CTA.  VEC: 16-byte accesses, the block in registers; else its elements are read twice.
template <typename T, bool VEC>
__global__ void __launch_bounds__(kThreads) tiles_kernel(const Fp8QuantArgs a, unsigned per_row)
{
    const int64_t row0 = (int64_t)(blockIdx.x / per_row) * kFp8Block;
    const int64_t col0 = (int64_t)(blockIdx.x % per_row) * kFp8Block;
    if constexpr (VEC) {
        constexpr int VW = Chunk<T>::kSize, kLanes = kFp8Block / VW, kRows = kThreads / kLanes, kN = kFp8Block / kRows;
        const int64_t col = col0 + threadIdx.x % kLanes * VW, row = row0 + threadIdx.x / kLanes;
        Chunk<T> x[kN];
        float m = 0.f;
#pragma unroll
        for (int i = 0; i < kN; ++i) {
            const bool in = col < a.D && row + i * kRows < a.rows;
            x[i].v = in ? __ldcs(reinterpret_cast<const uint4 *>((const T *)a.x + (row + i * kRows) * a.D + col))
                        : make_uint4(0u, 0u, 0u, 0u);
            m = fmaxf(m, x[i].most());
        }
        const float c = scale_of(block_max(m));
        const Unit unit(c);
        if (threadIdx.x == 0) a.scales[blockIdx.x] = c;
#pragma unroll
        for (int i = 0; i < kN; ++i)
            if (col < a.D && row + i * kRows < a.rows) x[i].put(a.q + (row + i * kRows) * a.D + col, unit);
    } else {
        const int64_t col = col0 + threadIdx.x % kFp8Block, last = min(row0 + kFp8Block, a.rows);
        float m = 0.f;
        if (col < a.D)
            for (int64_t r = row0 + threadIdx.x / kFp8Block; r < last; r += kThreads / kFp8Block)
                m = fmaxf(m, fabsf(to_f32(((const T *)a.x)[r * a.D + col])));
        const float c = scale_of(block_max(m));
        const Unit unit(c);
        if (threadIdx.x == 0) a.scales[blockIdx.x] = c;
        if (col < a.D)
            for (int64_t r = row0 + threadIdx.x / kFp8Block; r < last; r += kThreads / kFp8Block)
                a.q[r * a.D + col] = (unsigned char)pack_e4m3(both(to_f32(((const T *)a.x)[r * a.D + col])), unit);
    }
}

template <typename T>
cudaError_t run(const Fp8QuantArgs &a, cudaStream_t st)
{
    constexpr int VW = 16 / sizeof(T);
    const unsigned per_row = (unsigned)ceil_div(a.D, kFp8Block);
    const bool vec = a.D % VW == 0 && (((uintptr_t)a.x | (uintptr_t)a.q) & 15) == 0;
    if (a.block_rows > 1) {
        const unsigned grid = (unsigned)((a.rows + kFp8Block - 1) / kFp8Block * per_row);
        if (vec) tiles_kernel<T, true><<<grid, kThreads, 0, st>>>(a, per_row);
        else tiles_kernel<T, false><<<grid, kThreads, 0, st>>>(a, per_row);
        return cudaGetLastError();
    }
    const int64_t items = a.rows * per_row;
    const int64_t most = 152 * 8, ctas = (items * (vec ? kFp8Block / VW : 32) + kThreads - 1) / kThreads;
    const unsigned grid = (unsigned)(ctas < most ? ctas : most);
    if (vec && a.D % kFp8Block == 0) rows_kernel<T, true><<<grid, kThreads, 0, st>>>(a, items, per_row);
    else if (vec) rows_kernel<T, false><<<grid, kThreads, 0, st>>>(a, items, per_row);
    else rows_any_kernel<T><<<grid, kThreads, 0, st>>>(a, items, per_row);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_fp8_quantize(const Fp8QuantArgs &a, cudaStream_t st)
{
    return a.dt ? run<__nv_bfloat16>(a, st) : run<float>(a, st);
}

}  // namespace gdn
