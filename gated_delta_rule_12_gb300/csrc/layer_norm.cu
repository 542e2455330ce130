// layer_norm.cu -- layer norm over the last axis, forward and backward.
//
//     y = (x - mean) rstd w + b,   rstd = 1 / sqrt(mean((x - mean)^2) + eps)
// Backward, with xhat = (x - mean) rstd and u = dy w:
//     dx = rstd (u - mean(u) - xhat mean(u xhat)),   dw = sum_rows dy xhat,   db = sum_rows dy.
#include "common.cuh"
#include "kernels.h"

namespace gdn {
namespace {

constexpr int kThreads = 256;

// Sum over the block, the same bits in every thread.
__device__ __forceinline__ float block_sum(float v, float *sh)
{
    v = warp_sum(v);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = v;
    __syncthreads();
    float s = 0.f;
    for (int i = 0; i < kThreads / 32; ++i) s += sh[i];
    return s;
}

// One block per row; the variance from a second pass over the row's deviations.
template <typename T>
__global__ void __launch_bounds__(kThreads) norm_fwd_kernel(LayerNormArgs a)
{
    __shared__ float sh[kThreads / 32];
    for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
        const T *x = (const T *)a.x + r * a.D;
        float s = 0.f;
        for (int i = threadIdx.x; i < a.D; i += kThreads) s += to_f32(x[i]);
        const float mean = block_sum(s, sh) / a.D;
        s = 0.f;
        for (int i = threadIdx.x; i < a.D; i += kThreads) {
            const float d = to_f32(x[i]) - mean;
            s = fmaf(d, d, s);
        }
        const float rstd = 1.f / sqrtf(block_sum(s, sh) / a.D + a.eps);
        T *y = (T *)a.out + r * a.D;
        for (int i = threadIdx.x; i < a.D; i += kThreads) {
            const float xh = (to_f32(x[i]) - mean) * rstd;
            y[i] = from_f32<T>(fmaf(xh, a.weight ? a.weight[i] : 1.f, a.bias ? a.bias[i] : 0.f));
        }
        if (threadIdx.x == 0) {
            if (a.mean) a.mean[r] = mean;
            if (a.rstd) a.rstd[r] = rstd;
        }
    }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) norm_dx_kernel(LayerNormArgs a)
{
    __shared__ float sh[kThreads / 32];
    for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
        const T *x = (const T *)a.x + r * a.D, *dy = (const T *)a.dout + r * a.D;
        const float mean = a.mean[r], rstd = a.rstd[r];
        float s1 = 0.f, s2 = 0.f;
        for (int i = threadIdx.x; i < a.D; i += kThreads) {
            const float u = to_f32(dy[i]) * (a.weight ? a.weight[i] : 1.f);
            s1 += u;
            s2 = fmaf(u, (to_f32(x[i]) - mean) * rstd, s2);
        }
        const float c1 = block_sum(s1, sh) / a.D, c2 = block_sum(s2, sh) / a.D;
        T *dx = (T *)a.dx + r * a.D;
        for (int i = threadIdx.x; i < a.D; i += kThreads) {
            const float u = to_f32(dy[i]) * (a.weight ? a.weight[i] : 1.f);
            dx[i] = from_f32<T>(rstd * (u - c1 - (to_f32(x[i]) - mean) * rstd * c2));
        }
    }
}

constexpr int kRowSplits = 128;   // row ranges whose partial sums dw and db are joined from

// Partial sums of dw and db over one of kRowSplits row ranges, a thread per channel.
template <typename T>
__global__ void __launch_bounds__(kThreads) norm_dw_partial_kernel(LayerNormArgs a)
{
    const int ch = blockIdx.x * kThreads + threadIdx.x;
    if (ch >= a.D) return;
    const int64_t per = (a.rows + kRowSplits - 1) / kRowSplits, r0 = blockIdx.y * per;
    const int64_t r1 = r0 + per < a.rows ? r0 + per : a.rows;
    float sw = 0.f, sb = 0.f;
    for (int64_t r = r0; r < r1; ++r) {
        const float dy = to_f32(((const T *)a.dout)[r * a.D + ch]);
        sw = fmaf(dy, (to_f32(((const T *)a.x)[r * a.D + ch]) - a.mean[r]) * a.rstd[r], sw);
        sb += dy;
    }
    float *part = (float *)a.workspace + (int64_t)blockIdx.y * 2 * a.D;
    part[ch] = sw;
    part[a.D + ch] = sb;
}

__global__ void __launch_bounds__(kThreads) norm_dw_join_kernel(LayerNormArgs a)
{
    const int ch = blockIdx.x * kThreads + threadIdx.x;
    if (ch >= a.D) return;
    float sw = 0.f, sb = 0.f;
    for (int s = 0; s < kRowSplits; ++s) {
        sw += ((const float *)a.workspace)[(int64_t)s * 2 * a.D + ch];
        sb += ((const float *)a.workspace)[(int64_t)s * 2 * a.D + a.D + ch];
    }
    if (a.dweight) a.dweight[ch] = sw;
    if (a.dbias) a.dbias[ch] = sb;
}

template <typename T>
cudaError_t bwd(const LayerNormArgs &a, cudaStream_t st)
{
    const unsigned blocks = (unsigned)(a.rows < 152 * 8 ? a.rows : 152 * 8);
    if (a.dx && blocks) norm_dx_kernel<T><<<blocks, kThreads, 0, st>>>(a);
    if (a.dweight || a.dbias) {
        norm_dw_partial_kernel<T><<<dim3(ceil_div(a.D, kThreads), kRowSplits), kThreads, 0, st>>>(a);
        norm_dw_join_kernel<<<ceil_div(a.D, kThreads), kThreads, 0, st>>>(a);
    }
    return cudaGetLastError();
}

}  // namespace

size_t layer_norm_bwd_workspace_bytes(int64_t, int D, int) { return align256((size_t)kRowSplits * 2 * D * 4); }

cudaError_t launch_layer_norm_fwd(const LayerNormArgs &a, cudaStream_t st)
{
    const unsigned blocks = (unsigned)(a.rows < 152 * 8 ? a.rows : 152 * 8);
    if (a.dt) norm_fwd_kernel<__nv_bfloat16><<<blocks, kThreads, 0, st>>>(a);
    else norm_fwd_kernel<float><<<blocks, kThreads, 0, st>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_layer_norm_bwd(const LayerNormArgs &a, cudaStream_t st)
{
    return a.dt ? bwd<__nv_bfloat16>(a, st) : bwd<float>(a, st);
}

}  // namespace gdn
