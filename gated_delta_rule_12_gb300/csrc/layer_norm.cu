// layer_norm.cu -- layer norm over the last axis, forward and backward.
//
//     y = (x - mean) rstd w + b,   rstd = 1 / sqrt(mean((x - mean)^2) + eps)
// Backward, with xhat = (x - mean) rstd and u = dy w:
//     dx = rstd (u - mean(u) - xhat mean(u xhat)),   dw = sum_rows dy xhat,   db = sum_rows dy.
//
// Bound by memory: x and y forward; dy, x and dx backward.  A team of threads holds a row in registers, so each row is
// read once; the variance comes from the deviations in registers.  A thread keeps the same columns for every row of
// its team: w and b are read once a thread, and dw and db gather in registers, join over the CTA's teams in shared
// memory and leave one partial row a CTA, which a second kernel adds up.  Rows come up to four ahead through asynchronous
// copies: 32 KB of them in flight on an SM, as registers one row ahead allow, held the backward pass to 3.9 TB/s and the
// norm over heads (131072 x 128) to 2.6.  (Where two stages do not fit, backward with fp32 rows beyond 11264 elements, a
// row's copies overlap nothing.)  Rows of more than 16384 elements go through kernels that read them again, element by
// element (2000 x 32768 fp32 forward 225 us, 0.35 of the copy rate).
// Rows of other lengths than 16-byte accesses fit go by the 16-byte chunks that they lie in (48841 x 687 bf16: forward
// 32 us, backward 54 us; element by element 93 and 173), unless their tensors start elsewhere.
//
// Measured (GB300, bf16, device time): forward 8192 x 2048 14.8 us (4.5 TB/s); backward 25.7 us, 131072 x 128 backward
// 24.2 us (3.9 and 4.2 TB/s), of which about 3 us are the second kernel and the gap before it.
#include "common.cuh"
#include "kernels.h"
#include "pairs.cuh"

namespace gdn {
namespace {

// ---------------------------------------------------------------------------
// rows in registers
// ---------------------------------------------------------------------------

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

// TEAM: threads of a row's team where they are a part of a warp or a warp, 0 for `team` threads of several warps.
// MAX: most threads a CTA.
template <typename T, int VW, int NV, int TEAM, int MAX, int FIT>
__global__ void __launch_bounds__(MAX, MAX == 256 ? (NV * VW <= 8 ? 4 : NV * VW <= 16 ? 3 : 2) : 1)
rows_fwd_kernel(const LayerNormArgs a, int team)
{
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ __align__(16) float sh[2 * 32];
    using Rows = Ring<T, VW, NV, 1, MAX>;
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
    const T *next = (const T *)a.x + r * a.D - ph + lane * VW;
    T *y = (T *)a.out + r * a.D - ph + lane * VW;
    const int64_t step_d = step * a.D;
    auto load = [&](int stage, bool in) {
#pragma unroll
        for (int v = 0; v < NV; ++v)
            if constexpr (FIT == kShifted)
                ring.load_some(stage, 0, v, next + v * team * VW, in ? a.D + ph - (v * team + lane) * VW : 0);
            else
                ring.load(stage, 0, v, next + v * team * VW, in && live[v]);
        commit_copies();
        next += step_d;
    };
#pragma unroll
    for (int k = 0; k < kStages; ++k) load(k, r + k * step < a.rows);
    Pair w[NP], b[NP];
    uint32_t dead = 0;   // kShifted: the elements that are not the row's
#pragma unroll
    for (int i = 0; i < NP; ++i) {
        float wv[2], bv[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int v = (2 * i + k) / VW, c = (v * team + lane) * VW - ph + (2 * i + k) % VW;
            const bool is = live[v] && (FIT != kShifted || (c >= 0 && c < a.D));
            wv[k] = is && a.weight ? a.weight[c] : 1.f;
            bv[k] = is && a.bias ? a.bias[c] : 0.f;
            if (FIT == kShifted && !is) dead |= 1u << (2 * i + k);
        }
        w[i] = pair(wv[0], wv[1]);
        b[i] = pair(bv[0], bv[1]);
    }
    const int64_t rows_ahead = a.rows - kStages * step;
    int stage = 0;
    for (int64_t first = (int64_t)blockIdx.x * teams; first < a.rows; first += step, r += step, y += step_d) {
        Raw<T, VW> raw[NV];
        wait_copies<kStages - 1>();
        ring.read(stage, 0, raw);
        if (FIT == kShifted && lane == 0) raw[0].drop(ph);
        Pair x[NP], p = 0, q = 0;
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            x[i] = get_pair<T, VW, NV>(raw, i);
            if (i & 1) q = add2(q, x[i]);
            else p = add2(p, x[i]);
        }
        load(stage, r < rows_ahead);
        stage = (stage + 1) & (kStages - 1);
        float s[1] = {total(add2(p, q))};
        sum(s);
        const float mean = s[0] / (float)a.D;   // times 1 / D, a row of one value could miss its mean by an ulp, and x - mean 0
        p = q = 0;
#pragma unroll
        for (int i = 0; i < NP; ++i) x[i] = add2(x[i], both(-mean));
        if (FIT == kShifted && dead)
#pragma unroll
            for (int i = 0; i < NP; ++i) {
                float lo, hi;
                split(x[i], lo, hi);
                x[i] = pair(dead >> (2 * i) & 1 ? 0.f : lo, dead >> (2 * i + 1) & 1 ? 0.f : hi);
            }
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            if constexpr (VW == 1) {   // columns behind D take no part
                if (!live[2 * i + 1]) {
                    float lo, hi;
                    split(x[i], lo, hi);
                    x[i] = pair(live[2 * i] ? lo : 0.f, 0.f);
                }
            } else if constexpr (FIT != kShifted) {
                if (!live[2 * i / VW]) x[i] = 0;
            }
            if (i & 1) q = fma2(x[i], x[i], q);
            else p = fma2(x[i], x[i], p);
        }
        s[0] = total(add2(p, q));
        sum(s);
        const float rstd = inv_sqrt(fmaf(s[0], inv, a.eps));
        if (r < a.rows) {
#pragma unroll
            for (int i = 0; i < NP; ++i) x[i] = fma2(mul2(x[i], both(rstd)), w[i], b[i]);
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                const int c = (v * team + lane) * VW - ph;
                if (FIT == kShifted && live[v] && (c < 0 || c + VW > a.D))
                    put_some<T, VW>(y + v * team * VW, x, v, c, a.D);
                else if (live[v])
                    put<T, VW>(y + v * team * VW, x, v);
            }
            if (lane == 0) {
                if (a.mean) a.mean[r] = mean;
                if (a.rstd) a.rstd[r] = rstd;
            }
        }
    }
    wait_copies<0>();
}

// Stages of the backward kernel's ring for teams of more than 512 threads, 16 elements each: what fits beside the weight.
__host__ __device__ constexpr int again_stages(int stage_bytes, int threads)
{
    return 2 * stage_bytes + 64 * threads <= 226 * 1024 ? 2 : 1;
}

template <typename T, int VW, int NV, int TEAM, int MAX, int FIT>
__global__ void __launch_bounds__(MAX, MAX == 512 && NV * VW <= 8 ? 2 : 1) rows_bwd_kernel(const LayerNormArgs a, int team)
{
    extern __shared__ __align__(16) unsigned char smem[];   // the ring; at the end the sums
    __shared__ __align__(16) float sh[2 * 32 * 2];
    using Rows = Ring<T, VW, NV, 2, MAX>;
    // Teams of more than 512 threads have 64 registers each.  They read a row from the ring again behind its sums, and
    // the weight from shared memory, instead of keeping both (3581 x 9368 bf16: 76 us, 118 with them spilled; some
    // instances still spill 20 to 190 bytes).
    constexpr bool kAgain = MAX == 1024;
    const int stages = kAgain ? again_stages(Rows::stage_bytes(blockDim.x), blockDim.x) : Rows::kStages;
    const Rows ring(smem);
    if (TEAM) team = TEAM;
    TeamSum<TEAM, 2> sum(sh, team);
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
            if constexpr (FIT == kShifted) {
                const int left = in ? a.D + ph - (v * team + lane) * VW : 0;
                ring.load_some(stage, 0, v, x, left);
                ring.load_some(stage, 1, v, dy, left);
            } else {
                ring.load(stage, 0, v, x, in && live[v]);
                ring.load(stage, 1, v, dy, in && live[v]);
            }
        }
        commit_copies();
        at += step_d;
    };
    // the statistics come two rows ahead, in registers
    float2 stat[2];
    auto load_stat = [&](int64_t r) { return r < a.rows ? make_float2(__ldg(a.mean + r), __ldg(a.rstd + r)) : make_float2(0.f, 0.f); };
    stat[0] = load_stat(r);
    stat[1] = load_stat(r + step);
#pragma unroll
    for (int k = 0; k < stages; ++k) load(k, r + k * step < a.rows);
    Pair w[kAgain ? 1 : NP], dw[NP], db[NP];
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
        dw[i] = db[i] = 0;
    }
    const int64_t rows_ahead = a.rows - stages * step;
    int stage = 0;
    for (int64_t first = (int64_t)blockIdx.x * teams; first < a.rows; first += step, r += step, dx += step_d) {
        const float mean = stat[0].x, rstd = stat[0].y;
        stat[0] = stat[1];
        stat[1] = load_stat(r + 2 * step);
        // pairs of the accesses v to v + A - 1: x^ and u, with dy where the gradients' sums take it
        constexpr int A = kAgain ? (VW == 1 ? 2 : 1) : NV, P = A * VW / 2;
        Pair xh[P], u[P], p = 0, q = 0;
        auto take = [&](int v, bool sums) {
            Raw<T, VW> rx[A], rd[A];
            ring.read(stage, 0, rx, v);
            ring.read(stage, 1, rd, v);
            if (FIT == kShifted && lane == 0 && v == 0) {
                rx[0].drop(ph);
                rd[0].drop(ph);
            }
            // columns behind D: dy = 0, so u, its sums and the gradients' stay 0
#pragma unroll
            for (int i = 0; i < P; ++i) {
                const int k = v * VW / 2 + i;
                const Pair dy = get_pair<T, VW, A>(rd, i);
                xh[i] = mul2(add2(get_pair<T, VW, A>(rx, i), both(-mean)), both(rstd));
                if constexpr (kAgain) u[i] = mul2(dy, w_row[k * blockDim.x]);
                else u[i] = mul2(dy, w[k]);
                if (sums) {
                    p = add2(p, u[i]);
                    q = fma2(u[i], xh[i], q);
                    dw[k] = fma2(dy, xh[i], dw[k]);
                    db[k] = add2(db[k], dy);
                }
            }
        };
        if constexpr (!kAgain) wait_copies<Rows::kStages - 1>();
        else if (stages == 2) wait_copies<1>();
        else wait_copies<0>();
#pragma unroll
        for (int v = 0; v < NV; v += A) take(v, true);
        if (!kAgain) load(stage, r < rows_ahead);
        float s[2] = {total(p), total(q)};
        sum(s);
        const float c1 = s[0] * inv, c2 = s[1] * inv;
        const bool write = a.dx && r < a.rows;
        if (kAgain || write) {
#pragma unroll
            for (int v0 = 0; v0 < NV; v0 += A) {
                if constexpr (kAgain) take(v0, false);
#pragma unroll
                for (int i = 0; i < P; ++i)
                    u[i] = mul2(both(rstd), add2(u[i], fma2(xh[i], both(-c2), both(-c1))));
#pragma unroll
                for (int v = 0; v < A; ++v) {
                    const int c = ((v0 + v) * team + lane) * VW - ph;
                    T *to = dx + (v0 + v) * team * VW;
                    if (!write || !live[v0 + v]) continue;
                    if (FIT == kShifted && (c < 0 || c + VW > a.D)) put_some<T, VW>(to, u, v, c, a.D);
                    else put<T, VW>(to, u, v);
                }
            }
        }
        if (kAgain) load(stage, r < rows_ahead);
        stage = (stage + 1) & (stages - 1);
    }
    // the CTA's teams: those of a warp by shuffles, where they have the same columns, then one row [dw | db] a warp or team in shared memory, in order
    wait_copies<0>();
    if (!a.dweight && !a.dbias) return;
    __syncthreads();
    float *joined = reinterpret_cast<float *>(smem);
    const int own = FIT != kShifted && TEAM && TEAM < 32 ? 32 : team, rows = blockDim.x / own;
#pragma unroll
    for (int i = 0; i < NP; ++i) {
        float g[4];
        split(dw[i], g[0], g[1]);
        split(db[i], g[2], g[3]);
#pragma unroll
        for (int o = FIT != kShifted && TEAM ? TEAM : 32; o < 32; o *= 2)
#pragma unroll
            for (int k = 0; k < 4; ++k) g[k] += __shfl_xor_sync(0xffffffffu, g[k], o);
        if (threadIdx.x % own == lane)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int v = (2 * i + (k & 1)) / VW, c = (v * team + lane) * VW - ph + (2 * i + (k & 1)) % VW;
                if (live[v] && (FIT != kShifted || (c >= 0 && c < a.D))) joined[((threadIdx.x / own) * 2 + (k >> 1)) * a.D + c] = g[k];
            }
    }
    __syncthreads();
    float *part = (float *)a.workspace + (int64_t)blockIdx.x * 2 * a.D;
    for (int i = threadIdx.x; i < 2 * a.D; i += blockDim.x) {
        float t = joined[i];
        for (int k = 1; k < rows; ++k) t += joined[k * 2 * a.D + i];
        part[i] = t;
    }
}

// Adds up `parts` partial rows [dw | db]: 32 columns a block, every eighth row a warp, in order.
__global__ void __launch_bounds__(256) join_kernel(const LayerNormArgs a, int parts)
{
    __shared__ float sh[8][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t c = (int64_t)blockIdx.x * 32 + lane, n = 2 * (int64_t)a.D;
    asm volatile("griddepcontrol.wait;" ::: "memory");   // launched beside the kernel that writes the partial rows
    float s = 0.f;
    if (c < n)
        for (int p = warp; p < parts; p += 8) s += ((const float *)a.workspace)[p * n + c];
    sh[warp][lane] = s;
    __syncthreads();
    if (warp == 0 && c < n) {
        s = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) s += sh[i][lane];
        if (c < a.D) {
            if (a.dweight) a.dweight[c] = s;
        } else if (a.dbias) {
            a.dbias[c - a.D] = s;
        }
    }
}

// ---------------------------------------------------------------------------
// longer rows: a CTA a row, read again for every pass
// ---------------------------------------------------------------------------

constexpr int kThreads = 256;
constexpr int kRowSplits = 32;    // row ranges whose partial sums dw and db are joined from

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

template <typename T>
__global__ void __launch_bounds__(kThreads) long_fwd_kernel(const LayerNormArgs a)
{
    __shared__ float sh[kThreads / 32];
    const unsigned D = a.D;   // i + kThreads may pass 2^31
    for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
        const T *x = (const T *)a.x + r * a.D;
        float s = 0.f;
        for (unsigned i = threadIdx.x; i < D; i += kThreads) s += to_f32(x[i]);
        const float mean = block_sum(s, sh) / a.D;
        s = 0.f;
        for (unsigned i = threadIdx.x; i < D; i += kThreads) {
            const float d = to_f32(x[i]) - mean;
            s = fmaf(d, d, s);
        }
        const float rstd = 1.f / sqrtf(block_sum(s, sh) / a.D + a.eps);
        T *y = (T *)a.out + r * a.D;
        for (unsigned i = threadIdx.x; i < D; i += kThreads) {
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
__global__ void __launch_bounds__(kThreads) long_dx_kernel(const LayerNormArgs a)
{
    __shared__ float sh[kThreads / 32];
    const unsigned D = a.D;   // i + kThreads may pass 2^31
    for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
        const T *x = (const T *)a.x + r * a.D, *dy = (const T *)a.dout + r * a.D;
        const float mean = a.mean[r], rstd = a.rstd[r];
        float s1 = 0.f, s2 = 0.f;
        for (unsigned i = threadIdx.x; i < D; i += kThreads) {
            const float u = to_f32(dy[i]) * (a.weight ? a.weight[i] : 1.f);
            s1 += u;
            s2 = fmaf(u, (to_f32(x[i]) - mean) * rstd, s2);
        }
        const float c1 = block_sum(s1, sh) / a.D, c2 = block_sum(s2, sh) / a.D;
        T *dx = (T *)a.dx + r * a.D;
        for (unsigned i = threadIdx.x; i < D; i += kThreads) {
            const float u = to_f32(dy[i]) * (a.weight ? a.weight[i] : 1.f);
            dx[i] = from_f32<T>(rstd * (u - c1 - (to_f32(x[i]) - mean) * rstd * c2));
        }
    }
}

// Partial sums of dw and db over one of kRowSplits row ranges, a thread per channel.
template <typename T>
__global__ void __launch_bounds__(kThreads) long_dw_kernel(const LayerNormArgs a)
{
    const unsigned ch = blockIdx.x * kThreads + threadIdx.x;   // may pass 2^31
    if (ch >= (unsigned)a.D) return;
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

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

constexpr int kMost = 16384;   // elements of a row that 1024 threads hold

struct Shape { int team, wide; };   // threads a row; 0: `few` accesses each, 1: `many`, 2: three quarters of many

// The smallest team, whole warps up to 1024 threads, that can take the row at `many` accesses a thread; a part of a
// warp, or a warp, at `few` where that is enough.  (Powers of two alone: 8192 x 2049 bf16 35 us forward, 39.6
// backward; whole warps 28 and 29.8.)  8192 x 2048 bf16: forward 32 elements a thread 14.8 us, 16
// elements 15.5, 8 elements 19.8; backward, whose dw and db take twice as many registers, 16 elements 25.2 us,
// 8 elements 29.4, 32 elements (spilling) 51.
Shape shape(int D, int vw, int few, int many)
{
    const int nvec = ceil_div(D, vw);
    for (int g = 8; g <= 32; g *= 2)
        if (nvec <= g * few) return {g, 0};
    return {ceil_div(ceil_div(nvec, many), 32) * 32, 1};
}

template <typename T, int VW, int NV, int TEAM, int MAX, int FIT>
cudaError_t run_fwd(const LayerNormArgs &a, int team, cudaStream_t st)
{
    // a team of several warps is a CTA of its own
    const int threads = team > 256 ? team : 256 / team * team, smem = Ring<T, VW, NV, 1, MAX>::bytes(threads);
    const int64_t ctas = (a.rows + threads / team - 1) / (threads / team);
    const int most = kSMs * (threads > 256 ? 1 : (NV * VW <= 8 ? 4 : NV * VW <= 16 ? 3 : 2) * 256 / threads);
    if (smem > 32 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(rows_fwd_kernel<T, VW, NV, TEAM, MAX, FIT>,
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
    }
    rows_fwd_kernel<T, VW, NV, TEAM, MAX, FIT><<<(unsigned)(ctas < most ? ctas : most), threads, smem, st>>>(a, team);
    return cudaGetLastError();
}

// CTAs of 512 threads that an SM holds in the backward kernel: two where a thread has 8 elements or fewer.
int bwd_ctas(int D) { return D <= 256 ? 2 * kSMs : kSMs; }

cudaError_t launch_join(const LayerNormArgs &a, int parts, cudaStream_t st)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((2 * (int64_t)a.D + 31) / 32));
    cfg.blockDim = dim3(256);
    cfg.stream = st;
    cudaLaunchAttribute at = {};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, join_kernel, a, parts);
}

template <typename T, int VW, int NV, int TEAM, int MAX, int FIT>
cudaError_t run_bwd(const LayerNormArgs &a, int team, cudaStream_t st)
{
    const int threads = MAX / team * team;
    const int64_t ctas = (a.rows + threads / team - 1) / (threads / team);
    const int most = bwd_ctas(a.D), grid = (int)(ctas < most ? (ctas > 0 ? ctas : 1) : most);
    const bool sums = a.dweight || a.dbias;
    const int own = FIT != kShifted && team < 32 ? 32 : team, joined = sums ? threads / own * 2 * a.D * 4 : 0;
    using Rows = Ring<T, VW, NV, 2, MAX>;
    const int stage = Rows::stage_bytes(threads);
    const int ring = MAX == 1024 ? again_stages(stage, threads) * stage + 64 * threads : Rows::bytes(threads), smem = joined > ring ? joined : ring;
    if (smem > 32 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(rows_bwd_kernel<T, VW, NV, TEAM, MAX, FIT>,
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
    }
    rows_bwd_kernel<T, VW, NV, TEAM, MAX, FIT><<<grid, threads, smem, st>>>(a, team);
    const cudaError_t e = cudaGetLastError();
    return e != cudaSuccess || !sums ? e : launch_join(a, grid, st);
}

template <typename T, int VW, bool BWD, bool SHIFTED>
cudaError_t run(const LayerNormArgs &a, cudaStream_t st)
{
    constexpr int few = VW == 1 ? 4 : 8 / VW, many = VW == 1 ? 16 : (BWD ? 16 : 32) / VW;
    Shape s = shape(SHIFTED ? a.D + VW - 1 : a.D, VW, few, many);
    if constexpr (!BWD) {
        // 24 elements a thread where that leaves fewer threads idle (20000 x 1536 bf16 20 us, 32 elements 24; 8192 x
        // 2049 21.5 and 28; within 5 % it pays less: 3581 x 9368 35 and 33.5), and for shifted fp32 rows, which spill
        // with 32, unless many more are idle (8192 x 2047 26 and 42)
        const Shape t = shape(SHIFTED ? a.D + VW - 1 : a.D, VW, few, many * 3 / 4);
        const float most = SHIFTED && sizeof(T) == 4 ? 1.25f : 0.95f;
        if (t.wide && t.team <= 512 && t.team * 3 < most * (s.team * 4)) s = {t.team, 2};
    }
    const bool full = !SHIFTED && VW > 1 && a.D == s.team * VW * (s.wide == 2 ? many * 3 / 4 : s.wide ? many : few);
#define GDN_NORM1(NV, TEAM, FMAX, BMAX, FIT) \
    if constexpr (BWD) return run_bwd<T, VW, NV, TEAM, BMAX, FIT>(a, s.team, st); \
    else return run_fwd<T, VW, NV, TEAM, FMAX, FIT>(a, s.team, st)
#define GDN_NORM(NV, TEAM, FMAX, BMAX) \
    do { \
        if constexpr (SHIFTED) { GDN_NORM1(NV, TEAM, FMAX, BMAX, kShifted); } \
        if constexpr (VW > 1 && !SHIFTED) \
            if (full) { GDN_NORM1(NV, TEAM, FMAX, BMAX, kFull); } \
        if constexpr (!SHIFTED) { GDN_NORM1(NV, TEAM, FMAX, BMAX, kPartial); } \
    } while (0)
    if (s.team == 8) GDN_NORM(few, 8, 256, 512);
    if (s.team == 16) GDN_NORM(few, 16, 256, 512);
    if (s.team == 32 && !s.wide) GDN_NORM(few, 32, 256, 512);
    if constexpr (!BWD) {
        if (s.wide == 2 && s.team == 32) GDN_NORM(many * 3 / 4, 32, 256, 512);
        if (s.wide == 2 && s.team <= 256) GDN_NORM(many * 3 / 4, 0, 256, 512);
        if (s.wide == 2) GDN_NORM(many * 3 / 4, 0, 512, 512);
        if (s.team > 32 && s.team <= 256) GDN_NORM(many, 0, 256, 512);
    }
    if (s.team == 32) GDN_NORM(many, 32, 256, 512);
    if constexpr (BWD || VW == 1)
        if (s.team > 512) GDN_NORM(many, 0, 1024, 1024);
    GDN_NORM(many, 0, 512, 512);
#undef GDN_NORM
#undef GDN_NORM1
}

template <typename T, bool BWD>
cudaError_t run_rows(const LayerNormArgs &a, cudaStream_t st)
{
    constexpr int VW = 16 / sizeof(T);
    const uintptr_t starts = (uintptr_t)a.x | (uintptr_t)a.out | (uintptr_t)a.dout | (uintptr_t)a.dx;
    if ((starts & 15) == 0 && a.D % VW == 0) return run<T, VW, BWD, false>(a, st);
    if ((starts & 15) == 0 && a.D + VW - 1 <= kMost) return run<T, VW, BWD, true>(a, st);
    if constexpr (sizeof(T) == 2)
        if ((starts & 3) == 0 && a.D % 2 == 0) return run<T, 2, BWD, false>(a, st);
    return run<T, 1, BWD, false>(a, st);
}

template <typename T>
cudaError_t fwd(const LayerNormArgs &a, cudaStream_t st)
{
    if (a.D > kMost) {
        long_fwd_kernel<T><<<(unsigned)(a.rows < kSMs * 8 ? a.rows : kSMs * 8), kThreads, 0, st>>>(a);
        return cudaGetLastError();
    }
    return run_rows<T, false>(a, st);
}

template <typename T>
cudaError_t bwd(const LayerNormArgs &a, cudaStream_t st)
{
    if (a.D <= kMost) return run_rows<T, true>(a, st);
    const unsigned blocks = (unsigned)(a.rows < kSMs * 8 ? a.rows : kSMs * 8);
    // dx may lie over dout, so the sums over rows read dout first
    cudaError_t e = cudaSuccess;
    if (a.dweight || a.dbias) {
        long_dw_kernel<T><<<dim3(ceil_div(a.D, kThreads), kRowSplits), kThreads, 0, st>>>(a);
        e = cudaGetLastError();
        if (e == cudaSuccess) e = launch_join(a, kRowSplits, st);
    }
    if (e != cudaSuccess || !a.dx || !blocks) return e;
    long_dx_kernel<T><<<blocks, kThreads, 0, st>>>(a);
    return cudaGetLastError();
}

}  // namespace

size_t layer_norm_bwd_workspace_bytes(int64_t, int D, int)
{
    return align256((size_t)(D > kMost ? kRowSplits : bwd_ctas(D)) * 2 * D * 4);
}

cudaError_t launch_layer_norm_fwd(const LayerNormArgs &a, cudaStream_t st)
{
    return a.dt ? fwd<__nv_bfloat16>(a, st) : fwd<float>(a, st);
}

cudaError_t launch_layer_norm_bwd(const LayerNormArgs &a, cudaStream_t st)
{
    return a.dt ? bwd<__nv_bfloat16>(a, st) : bwd<float>(a, st);
}

}  // namespace gdn
