// gated_scan.cu -- per-channel gated linear recurrence: forward, backward and single-token step.
//
//     h_t = a_t h_{t-1} + c_t x_t,   a = exp(g),   c = 1, or 1 - a with the input gate.
//
// Backward, with e_t = dL/dh_{t-1} (through h_t), a scan from the end of the same form:
//     dH_t = dout_t + e_{t+1},   e_t = a_t dH_t,   e_{len} = dfinal,
//     dx_t = c_t dH_t,           dg_t = a_t dH_t (h_{t-1} [- x_t with the input gate]),   dinit = e_0.
#include "common.cuh"
#include "kernels.h"

namespace gdn {
namespace {

__device__ __forceinline__ void span(const GatedScanArgs &a, int n, int64_t &tok0, int &len)
{
    if (a.cu) {
        const int lo = __ldg(a.cu + n);
        tok0 = lo;
        len = __ldg(a.cu + n + 1) - lo;
    } else {
        tok0 = (int64_t)n * a.T;
        len = a.T;
    }
}

// One thread per (sequence, channel), one step after the other.
template <typename T, bool GATE>
__global__ void __launch_bounds__(128) scan_fwd_kernel(GatedScanArgs a)
{
    const int ch = blockIdx.x * blockDim.x + threadIdx.x;
    if (ch >= a.D) return;
    for (int n = blockIdx.y; n < a.N; n += gridDim.y) {
        int64_t tok0;
        int len;
        span(a, n, tok0, len);
        float h = a.init_state ? a.init_state[(int64_t)n * a.D + ch] : 0.f;
        for (int t = 0; t < len; ++t) {
            const int64_t i = (tok0 + t) * a.D + ch;
            const float g = to_f32(((const T *)a.g)[i]), x = to_f32(((const T *)a.x)[i]);
            h = fmaf(expf(g), h, GATE ? -expm1f(g) * x : x);
            ((T *)a.out)[i] = from_f32<T>(h);
        }
        if (a.final_state) a.final_state[(int64_t)n * a.D + ch] = h;
    }
}

template <typename T, bool GATE>
__global__ void __launch_bounds__(128) scan_bwd_kernel(GatedScanArgs a)
{
    const int ch = blockIdx.x * blockDim.x + threadIdx.x;
    if (ch >= a.D) return;
    for (int n = blockIdx.y; n < a.N; n += gridDim.y) {
        int64_t tok0;
        int len;
        span(a, n, tok0, len);
        const int64_t s = (int64_t)n * a.D + ch;
        float e = a.dfinal ? a.dfinal[s] : 0.f;
        for (int t = len - 1; t >= 0; --t) {
            const int64_t i = (tok0 + t) * a.D + ch;
            const float g = to_f32(((const T *)a.g)[i]), al = expf(g);
            float prev = t > 0 ? to_f32(((const T *)a.h)[i - a.D]) : (a.init_state ? a.init_state[s] : 0.f);
            const float dh = to_f32(((const T *)a.dout)[i]) + e;
            e = al * dh;
            if (GATE) prev -= to_f32(((const T *)a.x)[i]);
            ((T *)a.dx)[i] = from_f32<T>(GATE ? -expm1f(g) * dh : dh);
            ((T *)a.dg)[i] = from_f32<T>(e * prev);
        }
        if (a.dinit) a.dinit[s] = e;
    }
}

template <typename T, bool GATE>
__global__ void __launch_bounds__(256) scan_step_kernel(float *state, const T *x, const T *g, T *out, int64_t n)
{
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
        const float gv = to_f32(g[i]), xv = to_f32(x[i]);
        const float h = fmaf(expf(gv), state[i], GATE ? -expm1f(gv) * xv : xv);
        state[i] = h;
        out[i] = from_f32<T>(h);
    }
}

template <typename T, bool GATE>
cudaError_t fwd(const GatedScanArgs &a, cudaStream_t st)
{
    scan_fwd_kernel<T, GATE><<<dim3(ceil_div(a.D, 128), a.N < 65535 ? a.N : 65535), 128, 0, st>>>(a);
    return cudaGetLastError();
}

template <typename T, bool GATE>
cudaError_t bwd(const GatedScanArgs &a, cudaStream_t st)
{
    scan_bwd_kernel<T, GATE><<<dim3(ceil_div(a.D, 128), a.N < 65535 ? a.N : 65535), 128, 0, st>>>(a);
    return cudaGetLastError();
}

template <typename T, bool GATE>
cudaError_t step(float *state, const void *x, const void *g, void *out, int64_t n, cudaStream_t st)
{
    const int64_t blocks = (n + 255) / 256;
    scan_step_kernel<T, GATE><<<(unsigned)(blocks < 152 * 8 ? blocks : 152 * 8), 256, 0, st>>>(
        state, (const T *)x, (const T *)g, (T *)out, n);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_gated_scan_fwd(const GatedScanArgs &a, cudaStream_t st)
{
    if (a.dt) return a.input_gate ? fwd<__nv_bfloat16, true>(a, st) : fwd<__nv_bfloat16, false>(a, st);
    return a.input_gate ? fwd<float, true>(a, st) : fwd<float, false>(a, st);
}

cudaError_t launch_gated_scan_bwd(const GatedScanArgs &a, cudaStream_t st)
{
    if (a.dt) return a.input_gate ? bwd<__nv_bfloat16, true>(a, st) : bwd<__nv_bfloat16, false>(a, st);
    return a.input_gate ? bwd<float, true>(a, st) : bwd<float, false>(a, st);
}

cudaError_t launch_gated_scan_step(float *state, const void *x, const void *g, void *out, int64_t n, int dt,
                                   int input_gate, cudaStream_t st)
{
    if (dt) return input_gate ? step<__nv_bfloat16, true>(state, x, g, out, n, st)
                              : step<__nv_bfloat16, false>(state, x, g, out, n, st);
    return input_gate ? step<float, true>(state, x, g, out, n, st) : step<float, false>(state, x, g, out, n, st);
}

}  // namespace gdn
