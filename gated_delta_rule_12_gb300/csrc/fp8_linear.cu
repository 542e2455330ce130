// fp8_linear.cu -- product of 8-bit operands with scales: out = x w', x [M, K] e4m3 with a scale for each 128 columns of a
// row, w [N, K] e4m3 with a scale for each 128 x 128 block, out bf16:
//     out_mn = sum_b xs_mb ws_{n / 128, b} sum_{k in block b} x_mk w_nk.
//
// This kernel runs on the CUDA cores, for K that is no multiple of 16 (rows that TMA cannot address) and tensors that start
// elsewhere than on 16-byte boundaries; the others take the tensor cores (fp8_linear_tc.cu).  Bound by the fp32 units: a
// 64 x 64 tile a CTA, the operands widened to fp32 on their way into shared memory.  Products of a block are summed by
// themselves, then scaled: e4m3 products are exact in fp32.
#include "common.cuh"
#include "kernels.h"

namespace gdn {
namespace {

constexpr int kTile = 64, kDepth = 32, kThreads = 256;

__device__ __forceinline__ float from_e4m3(unsigned char v)
{
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((unsigned short)v));
    float f;
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.f32.f16 %0, lo;\n\t}" : "=f"(f) : "r"(h));
    return f;
}

__global__ void __launch_bounds__(kThreads) simt_kernel(const Fp8LinearArgs a, int nt)
{
    __shared__ float xs[kDepth][kTile + 4], ws[kDepth][kTile + 4];
    const int row0 = (int)(blockIdx.x / nt) * kTile, col0 = (int)(blockIdx.x % nt) * kTile;
    const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
    const int blocks = (a.K + kFp8Block - 1) / kFp8Block;
    if (threadIdx.x == 0 && blockIdx.x == 0) *(unsigned *)a.workspace = kDevErrNone;
    float total[4][4] = {};
    for (int b = 0; b < blocks; ++b) {
        float acc[4][4] = {};
        const int64_t end = min((int64_t)(b + 1) * kFp8Block, (int64_t)a.K);
        for (int64_t k0 = (int64_t)b * kFp8Block; k0 < end; k0 += kDepth) {
            __syncthreads();
            for (int i = threadIdx.x; i < kTile * kDepth; i += kThreads) {
                const int k = i % kDepth, r = i / kDepth;
                const bool in_k = k0 + k < end;
                xs[k][r] = in_k && row0 + r < a.M ? from_e4m3(a.x[(int64_t)(row0 + r) * a.K + k0 + k]) : 0.f;
                ws[k][r] = in_k && col0 + r < a.N ? from_e4m3(a.w[(int64_t)(col0 + r) * a.K + k0 + k]) : 0.f;
            }
            __syncthreads();
#pragma unroll 8
            for (int k = 0; k < kDepth; ++k) {
                const float4 x = *reinterpret_cast<const float4 *>(&xs[k][ty * 4]);
                const float4 w = *reinterpret_cast<const float4 *>(&ws[k][tx * 4]);
                const float xv[4] = {x.x, x.y, x.z, x.w}, wv[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(xv[i], wv[j], acc[i][j]);
            }
        }
        const int col = min(col0 + tx * 4, a.N - 1);   // a 64-column tile lies in one block of 128
        const float wscale = a.ws[(int64_t)(col / kFp8Block) * blocks + b];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int row = min(row0 + ty * 4 + i, a.M - 1);
            const float scale = a.xs[(int64_t)row * blocks + b] * wscale;
#pragma unroll
            for (int j = 0; j < 4; ++j) total[i][j] = fmaf(acc[i][j], scale, total[i][j]);
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (row0 + ty * 4 + i < a.M && col0 + tx * 4 + j < a.N)
                ((__nv_bfloat16 *)a.out)[(int64_t)(row0 + ty * 4 + i) * a.N + col0 + tx * 4 + j] = __float2bfloat16_rn(total[i][j]);
}

}  // namespace

size_t fp8_linear_workspace_bytes(int, int, int) { return 256; }

cudaError_t launch_fp8_linear(const Fp8LinearArgs &a, cudaStream_t st)
{
    if (fp8_linear_tc_supported(a)) return launch_fp8_linear_tc(a, st);
    const int mt = ceil_div(a.M, kTile), nt = ceil_div(a.N, kTile);
    simt_kernel<<<(unsigned)((int64_t)mt * nt), kThreads, 0, st>>>(a, nt);
    return cudaGetLastError();
}

}  // namespace gdn
