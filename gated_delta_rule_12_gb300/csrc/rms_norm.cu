// rms_norm.cu -- root-mean-square norm over the last axis with the residual's addition: forward, forward with an output
// in 8 bits and its scales, backward.
//
//     s = x + r (rounded to the element type, as it is stored),  y = s rstd w,  rstd = 1 / sqrt(mean(s^2) + eps)
//     8 bits: q = e4m3(y / c), c = max(|y|, 2^-100) / 448 over each 128 columns of a row
// Backward, with xhat = s rstd and u = dy w:
//     ds = rstd (u - xhat mean(u xhat)) + dr,   dw = sum_rows dy xhat,  dr the gradient that comes to s from elsewhere.
//
// The norm is of the rounded s, so that a backward pass from the stored row meets the numbers of the forward pass.  Sums
// and statistics are fp32; y is rounded once, to the element type or, in units of its block's scale, to e4m3.
//
// Bound by memory.  Rows go through teams of threads as in the layer norm (rows.cuh): read once, held in registers, the
// next rows on their way.  One sum a row instead of the layer norm's two takes the forward pass to the copy rate.
//
// Measured (GB300, device time, 8192 x 2048 bf16): forward with the residual's addition 19.6 us (6.9 TB/s), with 8-bit output
// 18.8 us (6.3); backward with dr 26.4 us (5.1), of which about 2 are the join of dw.  fp32: 44.8 us (6.0), 37.0 (5.9), 45.5 (5.9).
#include "common.cuh"
#include "fp8.cuh"
#include "kernels.h"
#include "pairs.cuh"
#include "rows.cuh"

namespace gdn {
namespace {

using namespace rows;

template <typename T>
__device__ __forceinline__ Pair rounded(Pair p)
{
    if constexpr (sizeof(T) == 4) return p;
    float a, b;
    uint32_t w;
    split(p, a, b);
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(b), "f"(a));
    return pair(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

// RES: the residual is added and the sum stored.  Q8: 8-bit output; rows start on 16-byte boundaries then, and a
// block's columns are those of 16 bf16 or 32 fp32 threads of one access, or, where a team is less than a warp, the row.
template <typename T, int VW, int NV, int TEAM, int MAX, int FIT, bool RES, bool Q8>
__global__ void __launch_bounds__(MAX, MAX == 256 ? (NV * VW <= 8 ? 4 : NV * VW <= 16 ? 3 : 2) : 1)
rms_fwd_kernel(const RmsNormArgs a, int team)
{
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ __align__(16) float sh[2 * 32];
    using Rows = Ring<T, VW, NV, RES ? 2 : 1, MAX>;
    constexpr int kStages = Rows::kStages;
    const Rows ring(smem);
    if (TEAM) team = TEAM;
    TeamSum<TEAM, 1> sum(sh, team);
    constexpr int NP = NV * VW / 2;
    const int lane = threadIdx.x % team, teams = blockDim.x / team;
    const int64_t step = (int64_t)gridDim.x * teams;
    const float inv = 1.f / (float)a.D;
    // every team of a CTA goes through the same number of rows: the shuffles take whole warps
    int64_t r = (int64_t)blockIdx.x * teams + threadIdx.x / team;
    const int ph = FIT == kShifted ? (int)(r * a.D % VW) : 0;
    bool live[NV];
#pragma unroll
    for (int v = 0; v < NV; ++v) live[v] = FIT == kFull || (v * team + lane) * VW - ph < a.D;
    int64_t at = r * a.D - ph + lane * VW, next = at;
    const int64_t step_d = step * a.D;
    auto load = [&](int stage, bool in) {
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const T *x = (const T *)a.x + next + v * team * VW, *res = RES ? (const T *)a.residual + next + v * team * VW : x;
            if constexpr (FIT == kShifted) {
                const int left = in ? a.D + ph - (v * team + lane) * VW : 0;
                ring.load_some(stage, 0, v, x, left);
                if constexpr (RES) ring.load_some(stage, 1, v, res, left);
            } else {
                ring.load(stage, 0, v, x, in && live[v]);
                if constexpr (RES) ring.load(stage, 1, v, res, in && live[v]);
            }
        }
        commit_copies();
        next += step_d;
    };
#pragma unroll
    for (int k = 0; k < kStages; ++k) load(k, r + k * step < a.rows);
    Pair w[NP];
#pragma unroll
    for (int i = 0; i < NP; ++i) {
        float wv[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int v = (2 * i + k) / VW, c = (v * team + lane) * VW - ph + (2 * i + k) % VW;
            const bool is = live[v] && (FIT != kShifted || (c >= 0 && c < a.D));
            wv[k] = is && a.weight ? a.weight[c] : 1.f;
        }
        w[i] = pair(wv[0], wv[1]);
    }
    const int64_t rows_ahead = a.rows - kStages * step;
    int stage = 0;
    for (int64_t first = (int64_t)blockIdx.x * teams; first < a.rows; first += step, r += step, at += step_d) {
        Pair t[NP], p = 0, q = 0;
        wait_copies<kStages - 1>();
        {
            Raw<T, VW> raw[NV], more[RES ? NV : 1];
            ring.read(stage, 0, raw);
            if constexpr (RES) ring.read(stage, 1, more);
            if (FIT == kShifted && lane == 0) {
                raw[0].drop(ph);
                if constexpr (RES) more[0].drop(ph);
            }
            // columns that are not the row's read as zeros and stay zeros
#pragma unroll
            for (int i = 0; i < NP; ++i) {
                t[i] = get_pair<T, VW, NV>(raw, i);
                if constexpr (RES) t[i] = rounded<T>(add2(t[i], get_pair<T, VW, NV>(more, i)));
                if (i & 1) q = fma2(t[i], t[i], q);
                else p = fma2(t[i], t[i], p);
            }
        }
        load(stage, r < rows_ahead);
        stage = (stage + 1) & (kStages - 1);
        float s[1] = {total(add2(p, q))};
        sum(s);
        const float rstd = inv_sqrt(fmaf(s[0], inv, a.eps));
        const bool in = r < a.rows;
        if (RES && in) {
            T *to = (T *)a.residual_out + at;
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                const int c = (v * team + lane) * VW - ph;
                if (FIT == kShifted && live[v] && (c < 0 || c + VW > a.D)) put_some<T, VW>(to + v * team * VW, t, v, c, a.D);
                else if (live[v]) put<T, VW>(to + v * team * VW, t, v);
            }
        }
#pragma unroll
        for (int i = 0; i < NP; ++i) t[i] = mul2(mul2(t[i], both(rstd)), w[i]);
        if constexpr (Q8) {
            constexpr int kLanes = VW == 8 ? 16 : 32;            // a block's threads
            constexpr bool kOne = TEAM && TEAM < 32;             // the row is one block
            float most[NV];
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                most[v] = 0.f;
#pragma unroll
                for (int i = 0; i < VW / 2; ++i) most[v] = largest(t[v * VW / 2 + i], most[v]);
            }
            if constexpr (kOne)
#pragma unroll
                for (int v = 1; v < NV; ++v) most[0] = fmaxf(most[0], most[v]);
#pragma unroll
            for (int o = (kOne ? TEAM : kLanes) / 2; o > 0; o >>= 1)
#pragma unroll
                for (int v = 0; v < (kOne ? 1 : NV); ++v) most[v] = fmaxf(most[v], __shfl_xor_sync(0xffffffffu, most[v], o));
            const int blocks = (a.D + kFp8Block - 1) / kFp8Block;
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                const float c = scale_of(most[kOne ? 0 : v]);
                const Unit unit(c);
                if (!in || !live[v]) continue;
                unsigned char *to = (unsigned char *)a.out + at + v * team * VW;
                if constexpr (VW == 8)
                    *reinterpret_cast<uint2 *>(to) = make_uint2(pack_e4m3(t[4 * v], t[4 * v + 1], unit),
                                                                pack_e4m3(t[4 * v + 2], t[4 * v + 3], unit));
                else
                    *reinterpret_cast<uint32_t *>(to) = pack_e4m3(t[2 * v], t[2 * v + 1], unit);
                if (kOne ? lane == 0 && v == 0 : lane % kLanes == 0)
                    a.scales[r * blocks + (kOne ? 0 : (v * team + lane) / kLanes)] = c;
            }
        } else if (in) {
            T *y = (T *)a.out + at;
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                const int c = (v * team + lane) * VW - ph;
                if (FIT == kShifted && live[v] && (c < 0 || c + VW > a.D)) put_some<T, VW>(y + v * team * VW, t, v, c, a.D);
                else if (live[v]) put<T, VW>(y + v * team * VW, t, v);
            }
        }
        if (in && lane == 0 && a.rstd) a.rstd[r] = rstd;
    }
    wait_copies<0>();
}

// RES: dr is added to ds.
template <typename T, int VW, int NV, int TEAM, int MAX, int FIT, bool RES>
__global__ void __launch_bounds__(MAX, MAX == 512 && NV * VW <= 8 ? 2 : 1) rms_bwd_kernel(const RmsNormArgs a, int team)
{
    extern __shared__ __align__(16) unsigned char smem[];   // the ring; at the end the sums
    __shared__ __align__(16) float sh[2 * 32];
    // Teams of more than 512 threads read a row again behind its sum, as the layer norm's; dr, which is used only there,
    // they read from memory, as three tensors' rows of 16384 fp32 do not fit beside the weight.
    constexpr bool kAgain = MAX == 1024, kRing = RES && !kAgain;
    using Rows = Ring<T, VW, NV, kRing ? 3 : 2, MAX>;
    const int stages = kAgain ? again_stages(Rows::stage_bytes(blockDim.x), blockDim.x) : Rows::kStages;
    const Rows ring(smem);
    if (TEAM) team = TEAM;
    TeamSum<TEAM, 1> sum(sh, team);
    constexpr int NP = NV * VW / 2;
    const int lane = threadIdx.x % team, teams = blockDim.x / team;
    const int64_t step = (int64_t)gridDim.x * teams;
    const float inv = 1.f / (float)a.D;
    int64_t r = (int64_t)blockIdx.x * teams + threadIdx.x / team;
    const int ph = FIT == kShifted ? (int)(r * a.D % VW) : 0;
    bool live[NV];
#pragma unroll
    for (int v = 0; v < NV; ++v) live[v] = FIT == kFull || (v * team + lane) * VW - ph < a.D;
    int64_t at = r * a.D - ph + lane * VW;
    T *dx = (T *)a.dx + at;
    const int64_t step_d = step * a.D;
    auto load = [&](int stage, bool in) {
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const T *x = (const T *)a.x + at + v * team * VW, *dy = (const T *)a.dout + at + v * team * VW;
            const T *dr = kRing ? (const T *)a.dresidual + at + v * team * VW : x;
            if constexpr (FIT == kShifted) {
                const int left = in ? a.D + ph - (v * team + lane) * VW : 0;
                ring.load_some(stage, 0, v, x, left);
                ring.load_some(stage, 1, v, dy, left);
                if constexpr (kRing) ring.load_some(stage, 2, v, dr, left);
            } else {
                ring.load(stage, 0, v, x, in && live[v]);
                ring.load(stage, 1, v, dy, in && live[v]);
                if constexpr (kRing) ring.load(stage, 2, v, dr, in && live[v]);
            }
        }
        commit_copies();
        at += step_d;
    };
    // the statistics come two rows ahead, in registers
    float stat[2];
    auto load_stat = [&](int64_t r) { return r < a.rows ? __ldg(a.rstd + r) : 0.f; };
    stat[0] = load_stat(r);
    stat[1] = load_stat(r + step);
#pragma unroll
    for (int k = 0; k < stages; ++k) load(k, r + k * step < a.rows);
    Pair w[kAgain ? 1 : NP], dw[NP];
    Pair *w_row = reinterpret_cast<Pair *>(smem + stages * Rows::stage_bytes(blockDim.x)) + threadIdx.x;   // kAgain
#pragma unroll
    for (int i = 0; i < NP; ++i) {
        float wv[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int v = (2 * i + k) / VW, c = (v * team + lane) * VW - ph + (2 * i + k) % VW;
            const bool is = live[v] && (FIT != kShifted || (c >= 0 && c < a.D));
            wv[k] = is && a.weight ? a.weight[c] : 1.f;
        }
        if constexpr (kAgain) w_row[i * blockDim.x] = pair(wv[0], wv[1]);
        else w[i] = pair(wv[0], wv[1]);
        dw[i] = 0;
    }
    const int64_t rows_ahead = a.rows - stages * step;
    int stage = 0;
    for (int64_t first = (int64_t)blockIdx.x * teams; first < a.rows; first += step, r += step, dx += step_d) {
        const float rstd = stat[0];
        stat[0] = stat[1];
        stat[1] = load_stat(r + 2 * step);
        // pairs of the accesses v to v + A - 1: xhat and u, with dy where the gradient's sum takes it
        constexpr int A = kAgain ? 1 : NV, P = A * VW / 2;
        Pair xh[P], u[P], p = 0, q = 0;
        auto take = [&](int v, bool sums) {
            Raw<T, VW> rx[A], rd[A];
            ring.read(stage, 0, rx, v);
            ring.read(stage, 1, rd, v);
            if (FIT == kShifted && lane == 0 && v == 0) {
                rx[0].drop(ph);
                rd[0].drop(ph);
            }
            // columns that are not the row's: dy = 0 and x = 0, so u, its sum and the gradient's stay 0
#pragma unroll
            for (int i = 0; i < P; ++i) {
                const int k = v * VW / 2 + i;
                const Pair dy = get_pair<T, VW, A>(rd, i);
                xh[i] = mul2(get_pair<T, VW, A>(rx, i), both(rstd));
                if constexpr (kAgain) u[i] = mul2(dy, w_row[k * blockDim.x]);
                else u[i] = mul2(dy, w[k]);
                if (sums) {
                    if (i & 1) q = fma2(u[i], xh[i], q);
                    else p = fma2(u[i], xh[i], p);
                    dw[k] = fma2(dy, xh[i], dw[k]);
                }
            }
        };
        if constexpr (!kAgain) wait_copies<Rows::kStages - 1>();
        else if (stages == 2) wait_copies<1>();
        else wait_copies<0>();
#pragma unroll
        for (int v = 0; v < NV; v += A) take(v, true);
        float s[1] = {total(add2(p, q))};
        sum(s);
        const float c = s[0] * inv;
        const bool write = a.dx && r < a.rows;
        if (kAgain || write) {
#pragma unroll
            for (int v0 = 0; v0 < NV; v0 += A) {
                if constexpr (kAgain) take(v0, false);
                Raw<T, VW> rr[RES ? A : 1];
                if constexpr (kRing) ring.read(stage, 2, rr, v0);
                else if constexpr (RES) {
                    const int col = (v0 * team + lane) * VW - ph;
                    const T *dr = (const T *)a.dresidual + r * a.D + col;
#pragma unroll
                    for (int k = 0; k < Raw<T, VW>::kWords; ++k) rr[0].w[k] = 0u;
                    if (write && live[v0]) {
                        if (FIT != kShifted || (col >= 0 && col + VW <= a.D)) {
                            const uint4 q = *reinterpret_cast<const uint4 *>(dr);
                            rr[0].w[0] = q.x; rr[0].w[1] = q.y; rr[0].w[2] = q.z; rr[0].w[3] = q.w;
                        } else {
#pragma unroll
                            for (int j = 0; j < VW; ++j)
                                if (col + j >= 0 && col + j < a.D) {
                                    if constexpr (sizeof(T) == 4) rr[0].w[j] = __float_as_uint(dr[j]);
                                    else rr[0].w[j / 2] |= (uint32_t)__bfloat16_as_ushort(dr[j]) << (16 * (j & 1));
                                }
                        }
                    }
                }
#pragma unroll
                for (int i = 0; i < P; ++i) {
                    u[i] = fma2(xh[i], both(-c), u[i]);
                    if constexpr (RES) u[i] = fma2(both(rstd), u[i], get_pair<T, VW, A>(rr, i));
                    else u[i] = mul2(both(rstd), u[i]);
                }
#pragma unroll
                for (int v = 0; v < A; ++v) {
                    const int col = ((v0 + v) * team + lane) * VW - ph;
                    T *to = dx + (v0 + v) * team * VW;
                    if (!write || !live[v0 + v]) continue;
                    if (FIT == kShifted && (col < 0 || col + VW > a.D)) put_some<T, VW>(to, u, v, col, a.D);
                    else put<T, VW>(to, u, v);
                }
            }
        }
        load(stage, r < rows_ahead);
        stage = (stage + 1) & (stages - 1);
    }
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // the join, which waits for the rows all the same
    // the CTA's teams: those of a warp by shuffles, where they have the same columns, then one row a warp or team in shared memory, in order
    wait_copies<0>();
    if (!a.dweight) return;
    __syncthreads();
    float *joined = reinterpret_cast<float *>(smem);
    const int own = FIT != kShifted && TEAM && TEAM < 32 ? 32 : team, rows = blockDim.x / own;
#pragma unroll
    for (int i = 0; i < NP; ++i) {
        float g[2];
        split(dw[i], g[0], g[1]);
#pragma unroll
        for (int o = FIT != kShifted && TEAM ? TEAM : 32; o < 32; o *= 2)
#pragma unroll
            for (int k = 0; k < 2; ++k) g[k] += __shfl_xor_sync(0xffffffffu, g[k], o);
        if (threadIdx.x % own == lane)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int v = (2 * i + k) / VW, c = (v * team + lane) * VW - ph + (2 * i + k) % VW;
                if (live[v] && (FIT != kShifted || (c >= 0 && c < a.D))) joined[threadIdx.x / own * a.D + c] = g[k];
            }
    }
    __syncthreads();
    float *part = (float *)a.workspace + (int64_t)blockIdx.x * a.D;
    for (int i = threadIdx.x; i < a.D; i += blockDim.x) {
        float t = joined[i];
        for (int k = 1; k < rows; ++k) t += joined[k * a.D + i];
        part[i] = t;
    }
}

// Adds up `parts` partial rows: 32 columns a block, every eighth row a warp, in order.
__global__ void __launch_bounds__(256) rms_join_kernel(const float *part, float *dweight, int D, int parts)
{
    __shared__ float sh[8][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t c = (int64_t)blockIdx.x * 32 + lane;
    asm volatile("griddepcontrol.wait;" ::: "memory");   // launched beside the kernel that writes the partial rows
    float s = 0.f;
    if (c < D)
        for (int p = warp; p < parts; p += 8) s += part[(int64_t)p * D + c];
    sh[warp][lane] = s;
    __syncthreads();
    if (warp == 0 && c < D) {
        s = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) s += sh[i][lane];
        dweight[c] = s;
    }
}

// ---------------------------------------------------------------------------
// other rows (longer, or in tensors that start elsewhere): a CTA a row, read again for every pass
// ---------------------------------------------------------------------------

constexpr int kThreads = 256;
constexpr int kRowSplits = 32;    // row ranges whose partial sums dw is joined from

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

template <typename T, bool RES, bool Q8>
__global__ void __launch_bounds__(kThreads) any_fwd_kernel(const RmsNormArgs a)
{
    __shared__ float sh[kThreads / 32];
    const unsigned D = a.D;   // i + kThreads may pass 2^31
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
        const T *x = (const T *)a.x + r * a.D, *t = x;
        float s = 0.f;
        if (RES) {
            const T *res = (const T *)a.residual + r * a.D;
            T *to = (T *)a.residual_out + r * a.D;
            for (unsigned i = threadIdx.x; i < D; i += kThreads) {
                const T v = from_f32<T>(to_f32(x[i]) + to_f32(res[i]));
                to[i] = v;
                s = fmaf(to_f32(v), to_f32(v), s);
            }
            t = to;
        } else {
            for (unsigned i = threadIdx.x; i < D; i += kThreads) s = fmaf(to_f32(x[i]), to_f32(x[i]), s);
        }
        const float rstd = inv_sqrt(block_sum(s, sh) / a.D + a.eps);   // its barriers bring the stored sum to all threads
        if (Q8) {
            const unsigned blocks = (D + kFp8Block - 1) / kFp8Block;
            unsigned char *to = (unsigned char *)a.out + r * a.D;
            for (unsigned b = warp; b < blocks; b += kThreads / 32) {
                float y[4], most = 0.f;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const unsigned c = b * kFp8Block + j * 32 + lane;
                    y[j] = c < D ? to_f32(t[c]) * rstd * (a.weight ? a.weight[c] : 1.f) : 0.f;
                    most = fmaxf(most, fabsf(y[j]));
                }
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
                const float c = scale_of(most);
                const Unit unit(c);
                if (lane == 0) a.scales[r * blocks + b] = c;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const unsigned i = b * kFp8Block + j * 32 + lane;
                    if (i < D) to[i] = (unsigned char)pack_e4m3(both(y[j]), unit);
                }
            }
        } else {
            T *y = (T *)a.out + r * a.D;
            for (unsigned i = threadIdx.x; i < D; i += kThreads)
                y[i] = from_f32<T>(to_f32(t[i]) * rstd * (a.weight ? a.weight[i] : 1.f));
        }
        if (threadIdx.x == 0 && a.rstd) a.rstd[r] = rstd;
    }
}

// 8-bit output of rows that 16-byte accesses do not fit, up to 128 NB elements: a warp a row, which it holds in registers, four
// elements of a lane in each block.
template <typename T, bool RES, int NB>
__global__ void __launch_bounds__(128) warp_fp8_kernel(const RmsNormArgs a)
{
    const int lane = threadIdx.x & 31, blocks = (a.D + kFp8Block - 1) / kFp8Block;
    for (int64_t r = (int64_t)blockIdx.x * 4 + threadIdx.x / 32; r < a.rows; r += (int64_t)gridDim.x * 4) {
        const T *x = (const T *)a.x + r * a.D, *res = RES ? (const T *)a.residual + r * a.D : x;
        float t[4 * NB], s = 0.f;
#pragma unroll
        for (int i = 0; i < 4 * NB; ++i) t[i] = i * 32 + lane < a.D ? to_f32(x[i * 32 + lane]) : 0.f;
        if constexpr (RES) {
            float q[4 * NB];
#pragma unroll
            for (int i = 0; i < 4 * NB; ++i) q[i] = i * 32 + lane < a.D ? to_f32(res[i * 32 + lane]) : 0.f;
#pragma unroll
            for (int i = 0; i < 4 * NB; ++i) {
                const T v = from_f32<T>(t[i] + q[i]);
                if (i * 32 + lane < a.D) ((T *)a.residual_out + r * a.D)[i * 32 + lane] = v;
                t[i] = to_f32(v);
            }
        }
#pragma unroll
        for (int i = 0; i < 4 * NB; ++i) s = fmaf(t[i], t[i], s);
        const float rstd = inv_sqrt(warp_sum(s) / a.D + a.eps);
        unsigned char *to = (unsigned char *)a.out + r * a.D;
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            if (b >= blocks) break;
            float most = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int c = b * kFp8Block + j * 32 + lane;
                float &y = t[4 * b + j];
                y = c < a.D ? y * rstd * (a.weight ? a.weight[c] : 1.f) : 0.f;
                most = fmaxf(most, fabsf(y));
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
            const float c = scale_of(most);
            const Unit unit(c);
            if (lane == 0) a.scales[r * blocks + b] = c;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (b * kFp8Block + j * 32 + lane < a.D) to[b * kFp8Block + j * 32 + lane] = (unsigned char)pack_e4m3(both(t[4 * b + j]), unit);
        }
    }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) any_dx_kernel(const RmsNormArgs a)
{
    __shared__ float sh[kThreads / 32];
    const unsigned D = a.D;   // i + kThreads may pass 2^31
    for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
        const T *x = (const T *)a.x + r * a.D, *dy = (const T *)a.dout + r * a.D;
        const T *dr = a.dresidual ? (const T *)a.dresidual + r * a.D : nullptr;
        const float rstd = a.rstd[r];
        float s = 0.f;
        for (unsigned i = threadIdx.x; i < D; i += kThreads)
            s = fmaf(to_f32(dy[i]) * (a.weight ? a.weight[i] : 1.f), to_f32(x[i]) * rstd, s);
        const float c = block_sum(s, sh) / a.D;
        T *dx = (T *)a.dx + r * a.D;
        for (unsigned i = threadIdx.x; i < D; i += kThreads) {
            const float u = to_f32(dy[i]) * (a.weight ? a.weight[i] : 1.f);
            dx[i] = from_f32<T>(fmaf(rstd, fmaf(to_f32(x[i]) * rstd, -c, u), dr ? to_f32(dr[i]) : 0.f));
        }
    }
}

// Partial sums of dw over one of kRowSplits row ranges, a thread per channel.
template <typename T>
__global__ void __launch_bounds__(kThreads) any_dw_kernel(const RmsNormArgs a)
{
    const unsigned ch = blockIdx.x * kThreads + threadIdx.x;   // may pass 2^31
    if (ch >= (unsigned)a.D) return;
    const int64_t per = (a.rows + kRowSplits - 1) / kRowSplits, r0 = blockIdx.y * per;
    const int64_t r1 = r0 + per < a.rows ? r0 + per : a.rows;
    float sw = 0.f;
    for (int64_t r = r0; r < r1; ++r)
        sw = fmaf(to_f32(((const T *)a.dout)[r * a.D + ch]), to_f32(((const T *)a.x)[r * a.D + ch]) * a.rstd[r], sw);
    ((float *)a.workspace)[(int64_t)blockIdx.y * a.D + ch] = sw;
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

// The limit that every launch of a kernel sets, whatever it takes itself: another thread's launch may come between the two.
constexpr int kMostSmem = 226 * 1024;

template <typename T, int VW, int NV, int TEAM, int MAX, int FIT, bool RES, bool Q8>
cudaError_t run_fwd(const RmsNormArgs &a, int team, cudaStream_t st)
{
    // a team of several warps is a CTA of its own
    const int threads = team > 256 ? team : 256 / team * team, smem = Ring<T, VW, NV, RES ? 2 : 1, MAX>::bytes(threads);
    const int64_t ctas = (a.rows + threads / team - 1) / (threads / team);
    const int most = kSMs * (threads > 256 ? 1 : (NV * VW <= 8 ? 4 : NV * VW <= 16 ? 3 : 2) * 256 / threads);
    if (smem > 32 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(rms_fwd_kernel<T, VW, NV, TEAM, MAX, FIT, RES, Q8>,
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize, kMostSmem);
        if (e != cudaSuccess) return e;
    }
    rms_fwd_kernel<T, VW, NV, TEAM, MAX, FIT, RES, Q8><<<(unsigned)(ctas < most ? ctas : most), threads, smem, st>>>(a, team);
    return cudaGetLastError();
}

// CTAs of 512 threads that an SM holds in the backward kernel: two where a thread has 8 elements or fewer.
int bwd_ctas(int D) { return D <= 256 ? 2 * kSMs : kSMs; }

cudaError_t launch_join(const RmsNormArgs &a, int parts, cudaStream_t st)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(((int64_t)a.D + 31) / 32));
    cfg.blockDim = dim3(256);
    cfg.stream = st;
    cudaLaunchAttribute at = {};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, rms_join_kernel, (const float *)a.workspace, a.dweight, a.D, parts);
}

template <typename T, int VW, int NV, int TEAM, int MAX, int FIT, bool RES>
cudaError_t run_bwd(const RmsNormArgs &a, int team, cudaStream_t st)
{
    const int threads = MAX / team * team;
    const int64_t ctas = (a.rows + threads / team - 1) / (threads / team);
    const int most = bwd_ctas(a.D), grid = (int)(ctas < most ? (ctas > 0 ? ctas : 1) : most);
    const int own = FIT != kShifted && team < 32 ? 32 : team, joined = a.dweight ? threads / own * a.D * 4 : 0;
    using Rows = Ring<T, VW, NV, RES && MAX < 1024 ? 3 : 2, MAX>;
    const int stage = Rows::stage_bytes(threads);
    const int ring = MAX == 1024 ? again_stages(stage, threads) * stage + 64 * threads : Rows::bytes(threads);
    const int smem = joined > ring ? joined : ring;
    if (smem > 32 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(rms_bwd_kernel<T, VW, NV, TEAM, MAX, FIT, RES>,
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize, kMostSmem);
        if (e != cudaSuccess) return e;
    }
    rms_bwd_kernel<T, VW, NV, TEAM, MAX, FIT, RES><<<grid, threads, smem, st>>>(a, team);
    const cudaError_t e = cudaGetLastError();
    return e != cudaSuccess || !a.dweight ? e : launch_join(a, grid, st);
}

enum { kFwd, kQ8, kBwd };

template <typename T, int OP, bool SHIFTED, bool RES>
cudaError_t run(const RmsNormArgs &a, cudaStream_t st)
{
    constexpr bool BWD = OP == kBwd;
    constexpr int VW = 16 / sizeof(T), few = 8 / VW, many = (BWD ? 16 : 32) / VW;
    const int held = SHIFTED ? a.D + VW - 1 : a.D;
    Shape s = shape(held, VW, few, many);
    if constexpr (!BWD) {
        // 24 elements a thread where that leaves fewer threads idle, and for shifted fp32 rows, which spill with 32, as
        // in the layer norm
        const Shape t = shape(held, VW, few, many * 3 / 4);
        const float most = SHIFTED && sizeof(T) == 4 ? 1.25f : 0.95f;
        if (t.wide && t.team <= 512 && t.team * 3 < most * (s.team * 4)) s = {t.team, 2};
    }
    const bool full = !SHIFTED && a.D == s.team * VW * (s.wide == 2 ? many * 3 / 4 : s.wide ? many : few);
#define GDN_NORM1(NV, TEAM, FMAX, BMAX, FIT) \
    if constexpr (BWD) return run_bwd<T, VW, NV, TEAM, BMAX, FIT, RES>(a, s.team, st); \
    else return run_fwd<T, VW, NV, TEAM, FMAX, FIT, RES, OP == kQ8>(a, s.team, st)
#define GDN_NORM(NV, TEAM, FMAX, BMAX) \
    do { \
        if constexpr (SHIFTED) { GDN_NORM1(NV, TEAM, FMAX, BMAX, kShifted); } \
        else { \
            if (full) { GDN_NORM1(NV, TEAM, FMAX, BMAX, kFull); } \
            GDN_NORM1(NV, TEAM, FMAX, BMAX, kPartial); \
        } \
    } while (0)
    if (s.team == 8) GDN_NORM(few, 8, 256, 512);
    if (s.team == 16) GDN_NORM(few, 16, 256, 512);
    if (s.team == 32 && !s.wide) GDN_NORM(few, 32, 256, 512);
    if (s.team == 32 && s.wide == 1) GDN_NORM(many, 32, 256, 512);
    if constexpr (BWD) {
        if (s.team > 512) GDN_NORM(many, 0, 1024, 1024);
    } else {
        if (s.wide == 2 && s.team == 32) GDN_NORM(many * 3 / 4, 32, 256, 512);
        if (s.wide == 2 && s.team <= 256) GDN_NORM(many * 3 / 4, 0, 256, 512);
        if (s.wide == 2) GDN_NORM(many * 3 / 4, 0, 512, 512);
        if (s.team <= 256) GDN_NORM(many, 0, 256, 512);
    }
    GDN_NORM(many, 0, 512, 512);
#undef GDN_NORM
#undef GDN_NORM1
}

// Rows that a team holds, in tensors that start on 16-byte boundaries; with an 8-bit output the rows have to as well.
bool by_teams(const RmsNormArgs &a, const void *y)
{
    const uintptr_t starts = (uintptr_t)a.x | (uintptr_t)a.residual | (uintptr_t)a.residual_out | (uintptr_t)y |
                             (uintptr_t)a.dout | (uintptr_t)a.dresidual;
    const int vw = a.dt ? 8 : 4;
    return (starts & 15) == 0 && a.D <= kMost && (a.D % vw == 0 || (!a.scales && a.D + vw - 1 <= kMost));
}

template <typename T, bool RES>
cudaError_t fwd(const RmsNormArgs &a, cudaStream_t st)
{
    if (by_teams(a, a.out)) {
        if (a.scales) return run<T, kQ8, false, RES>(a, st);
        return a.D % (16 / (int)sizeof(T)) == 0 ? run<T, kFwd, false, RES>(a, st) : run<T, kFwd, true, RES>(a, st);
    }
    const unsigned grid = (unsigned)(a.rows < kSMs * 8 ? a.rows : kSMs * 8);
    // a warp a row: 40000 x 100 bf16 11 us, a CTA a row 47; 8192 x 2049 197 us, spilled, and 53
    if (a.scales && a.D <= 8 * kFp8Block) {
        const int64_t ctas = (a.rows + 3) / 4, most = kSMs * 16;
        const unsigned warps = (unsigned)(ctas < most ? ctas : most);
        if (a.D <= kFp8Block) warp_fp8_kernel<T, RES, 1><<<warps, 128, 0, st>>>(a);
        else if (a.D <= 4 * kFp8Block) warp_fp8_kernel<T, RES, 4><<<warps, 128, 0, st>>>(a);
        else warp_fp8_kernel<T, RES, 8><<<warps, 128, 0, st>>>(a);
        return cudaGetLastError();
    }
    if (a.scales) any_fwd_kernel<T, RES, true><<<grid, kThreads, 0, st>>>(a);
    else any_fwd_kernel<T, RES, false><<<grid, kThreads, 0, st>>>(a);
    return cudaGetLastError();
}

template <typename T, bool RES>
cudaError_t bwd(const RmsNormArgs &a, cudaStream_t st)
{
    if (by_teams(a, a.dx))
        return a.D % (16 / (int)sizeof(T)) == 0 ? run<T, kBwd, false, RES>(a, st) : run<T, kBwd, true, RES>(a, st);
    const unsigned blocks = (unsigned)(a.rows < kSMs * 8 ? a.rows : kSMs * 8);
    // dx may lie over dout, so the sums over rows read dout first
    cudaError_t e = cudaSuccess;
    if (a.dweight) {
        any_dw_kernel<T><<<dim3(ceil_div(a.D, kThreads), kRowSplits), kThreads, 0, st>>>(a);
        e = cudaGetLastError();
        if (e == cudaSuccess) e = launch_join(a, kRowSplits, st);
    }
    if (e != cudaSuccess || !a.dx || !blocks) return e;
    any_dx_kernel<T><<<blocks, kThreads, 0, st>>>(a);
    return cudaGetLastError();
}

}  // namespace

size_t rms_norm_bwd_workspace_bytes(int D) { return align256((size_t)(D > kMost ? kRowSplits : bwd_ctas(D)) * D * 4); }

cudaError_t launch_rms_norm_fwd(const RmsNormArgs &a, cudaStream_t st)
{
    if (a.residual) return a.dt ? fwd<__nv_bfloat16, true>(a, st) : fwd<float, true>(a, st);
    return a.dt ? fwd<__nv_bfloat16, false>(a, st) : fwd<float, false>(a, st);
}

cudaError_t launch_rms_norm_bwd(const RmsNormArgs &a, cudaStream_t st)
{
    if (a.dresidual) return a.dt ? bwd<__nv_bfloat16, true>(a, st) : bwd<float, true>(a, st);
    return a.dt ? bwd<__nv_bfloat16, false>(a, st) : bwd<float, false>(a, st);
}

}  // namespace gdn
