// linear_ce.cu -- softmax cross entropy of a linear head over a large vocabulary, with its gradient,
// without an [N, V] array of logits.
//
//     l_iv = h_i . w_v,   lse_i = log sum_v exp(l_iv),   loss_i = lse_i - l_{i,t_i}
//     G_iv = (exp(l_iv - lse_i) - [v = t_i]) dloss_i,    dh = G W,   dW = G^T h.
// A row whose target is outside [0, V) is ignored: loss, lse and its gradients are 0, and nothing that its h
// holds (NaN included) reaches dW.
//
// The log probabilities' calls (log_probs.cuh) take the same kernels, with the entropy's sum and a tile's best words, and
// with the entropy's gradient in G.
//
// These kernels run on the CUDA cores: fp32, and bf16 whose rows are no multiple of 16 bytes; other bf16 sizes take the
// tensor cores (linear_ce_tc.cu).  Bound by the fp32 units where there are tiles for all SMs.  Measured (GB300, device time, fp32):
// 512 x 512 x 4096 loss 72 us (30 TFLOP/s), log probabilities 74, with five alternatives 84; 255 x 1024 x 50257 with eight 794 us
// (33).  Gradients 0.68 ms and 8.8 ms (9 TFLOP/s): dh of a piece has 16 tiles at these sizes.
//
// Forward: each 128 x 128 tile of logits leaves one (max, sum of exponentials) pair a row, joined by a second
// kernel in the order of the tiles.  Backward: the vocabulary is taken in pieces; a piece's G is recomputed into
// the workspace, then read by the two products.  All sums run in a fixed order.
#include "common.cuh"
#include "kernels.h"
#include "log_probs.cuh"

namespace gdn {
namespace {

constexpr int kTile = 128, kDepth = 16, kThreads = 256;

struct CeWorkspace {
    size_t part;     // forward: float2 [N][tiles]   (max, sum) of each row over each 128 columns
    size_t at;       // forward: float [N]           the target's logit
    size_t best;     // log probabilities, forward: float2 [N][tiles][top]   a tile's best words, part being RowStat then
    size_t g;        // backward: float [N][piece]   G of one piece of the vocabulary
    size_t acc;      // backward: float [N][D]       dh so far
    size_t total;
    int tiles, piece;
};

// top: the best words of a log-probability call, -1 for the cross entropy
CeWorkspace layout(int N, int D, int V, bool backward, int top = -1)
{
    CeWorkspace w = {};
    size_t off = 0;
    w.tiles = ceil_div(V, kTile);
    if (!backward) {
        w.part = off; off = align256(off + (size_t)N * w.tiles * (top < 0 ? sizeof(float2) : sizeof(RowStat)));
        w.at = off;   off = align256(off + (size_t)N * 4);
        w.best = off; off = align256(off + (top > 0 ? (size_t)N * w.tiles * top * sizeof(float2) : 0));
    } else {
        // a piece's G in about 64 MB
        const int64_t fit = ((int64_t)16 << 20) / (N > 0 ? N : 1) / kTile;
        w.piece = (int)(fit < 1 ? 1 : fit > w.tiles ? w.tiles : fit) * kTile;
        w.g = off;    off = align256(off + (size_t)N * w.piece * 4);
        w.acc = off;  off = align256(off + (size_t)N * D * 4);
    }
    w.total = off;
    return w;
}

// A thread's 8 x 8 of a tile: rows and columns 4 ty + {0..3} and 64 more, so that both operands come from shared memory
// in 16-byte reads.
__device__ __forceinline__ int row_of(int i) { return (threadIdx.x >> 4) * 4 + (i & 3) + (i >> 2) * 64; }
__device__ __forceinline__ int col_of(int j) { return (threadIdx.x & 15) * 4 + (j & 3) + (j >> 2) * 64; }

// acc(m, n) = sum_k A(m, k) B(n, k) for one 128 x 128 tile.  The loaders give 0 outside their arrays.  AMN (BMN):
// neighbouring threads load along m (n), else along k.  The next 16 of K are loaded while these are multiplied.
template <bool AMN, bool BMN, class LoadA, class LoadB>
__device__ __forceinline__ void tile_product(LoadA la, LoadB lb, int64_t K, float (&acc)[8][8])
{
    __shared__ __align__(16) float as[2][kDepth][kTile + 4], bs[2][kDepth][kTile + 4];
    constexpr int E = kTile * kDepth / kThreads;
    const int tid = threadIdx.x;
    float ra[E], rb[E];
    auto load = [&](int64_t k0) {
#pragma unroll
        for (int i = 0; i < E; ++i) {
            const int e = tid + i * kThreads;
            const int am = AMN ? e % kTile : e / kDepth, ak = AMN ? e / kTile : e % kDepth;
            const int bn = BMN ? e % kTile : e / kDepth, bk = BMN ? e / kTile : e % kDepth;
            ra[i] = k0 + ak < K ? la(am, k0 + ak) : 0.f;
            rb[i] = k0 + bk < K ? lb(bn, k0 + bk) : 0.f;
        }
    };
    auto store = [&](int turn) {
#pragma unroll
        for (int i = 0; i < E; ++i) {
            const int e = tid + i * kThreads;
            as[turn][AMN ? e / kTile : e % kDepth][AMN ? e % kTile : e / kDepth] = ra[i];
            bs[turn][BMN ? e / kTile : e % kDepth][BMN ? e % kTile : e / kDepth] = rb[i];
        }
    };
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[i][j] = 0.f;
    load(0);
    store(0);
    __syncthreads();
    int turn = 0;
    for (int64_t k0 = 0; k0 < K; k0 += kDepth, turn ^= 1) {
        const bool more = k0 + kDepth < K;
        if (more) load(k0 + kDepth);
#pragma unroll
        for (int k = 0; k < kDepth; ++k) {
            float av[8], bv[8];
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                *reinterpret_cast<float4 *>(av + 4 * q) = *reinterpret_cast<const float4 *>(&as[turn][k][row_of(4 * q)]);
                *reinterpret_cast<float4 *>(bv + 4 * q) = *reinterpret_cast<const float4 *>(&bs[turn][k][col_of(4 * q)]);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j) acc[i][j] = fmaf(av[i], bv[j], acc[i][j]);
        }
        if (more) store(turn ^ 1);
        __syncthreads();
    }
}

__device__ __forceinline__ bool kept(const LinearCeArgs &a, int row)
{
    const int t = a.targets[row];
    return t >= 0 && t < a.V;
}

// Logits of rows row0 + blockIdx.y * 128 .. and columns v0 + blockIdx.x * 128 ..; kBack: G of the piece (kBackEnt: with the
// entropy's gradient), else the tile's (max, sum) of each row and the target's logit where the tile holds it (kStats: what
// the entropy takes, and the tile's best words too).
enum { kLoss, kBack, kStats, kBackEnt };

template <typename T, int MODE>
__global__ void __launch_bounds__(kThreads, 2) ce_logits_kernel(LinearCeArgs a, CeWorkspace ws, int v0, int cols, int row0,
                                                                LogProbsGrad grad, int top_k)
{
    const int m0 = row0 + blockIdx.y * kTile, n0 = v0 + blockIdx.x * kTile;
    const T *h = (const T *)a.h, *w = (const T *)a.w;
    // the device error word in front of the workspace: these kernels have nothing to report
    if (blockIdx.x == 0 && m0 == 0 && threadIdx.x == 0) *((unsigned *)a.workspace - 64) = kDevErrNone;
    float acc[8][8];
    tile_product<false, false>(
        [&](int m, int64_t k) { return m0 + m < a.N ? to_f32(h[(int64_t)(m0 + m) * a.D + k]) : 0.f; },
        [&](int n, int64_t k) { return n0 + n < a.V ? to_f32(w[(int64_t)(n0 + n) * a.D + k]) : 0.f; }, a.D, acc);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int row = m0 + row_of(i);
        const bool in = row < a.N;   // the same for the 16 lanes that share the row
        const int t = in ? a.targets[row] : -1;
        const bool keep = t >= 0 && t < a.V;
        if (MODE == kBackEnt) {
            if (!in) continue;
            const float lse = a.lse_in[row], da = a.dloss[row], de = grad.dentropy[row], entropy = grad.entropy[row];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int v = n0 + col_of(j);
                if (v - v0 >= cols) continue;
                const float z = acc[i][j] - lse, g = expf(z) * fmaf(de, fmaxf(z, -1e4f) + entropy, da);   // 0 times -inf is 0 here
                ((float *)((char *)a.workspace + ws.g))[(int64_t)row * cols + (v - v0)] = keep ? (v == t ? da : 0.f) - g : 0.f;
            }
        } else if (MODE == kBack) {
            if (!in) continue;
            const float lse = a.lse_in[row], dl = grad.sign * a.dloss[row];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int v = n0 + col_of(j);
                if (v - v0 >= cols) continue;
                const float p = expf(acc[i][j] - lse) - (v == t ? 1.f : 0.f);
                ((float *)((char *)a.workspace + ws.g))[(int64_t)row * cols + (v - v0)] = keep ? p * dl : 0.f;
            }
        } else {
            float top = -INFINITY, sum = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (n0 + col_of(j) < a.V) top = fmaxf(top, acc[i][j]);
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            const float base = isinf(top) ? 0.f : top;   // keeps infinities and NaN in the sum
            float u = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int v = n0 + col_of(j);
                if (v >= a.V) continue;
                const float d = acc[i][j] - base, e = expf(d);
                sum += e;
                if (MODE == kStats) u = fmaf(e, fmaxf(d, -1e4f), u);   // 0 times -inf is 0 here
                if (in && v == t) ((float *)((char *)a.workspace + ws.at))[row] = acc[i][j];
            }
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            if (MODE == kStats) {
#pragma unroll
                for (int o = 8; o > 0; o >>= 1) u += __shfl_xor_sync(0xffffffffu, u, o);
                const int64_t at = (int64_t)row * ws.tiles + blockIdx.x;
                int count = 0;
                // a word a turn, the best one left among the 16 lanes' (most tiles of a row have few of its best, but which
                // is known only behind them all)
                for (; count < top_k; ++count) {
                    float x = -INFINITY;
                    int word = INT32_MAX;
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        if (n0 + col_of(j) < a.V && acc[i][j] > x) {
                            x = acc[i][j];
                            word = n0 + col_of(j);
                        }
#pragma unroll
                    for (int o = 8; o > 0; o >>= 1) {
                        const float y = __shfl_xor_sync(0xffffffffu, x, o);
                        const int other = __shfl_xor_sync(0xffffffffu, word, o);
                        if (y > x || (y == x && other < word)) {
                            x = y;
                            word = other;
                        }
                    }
                    if (word == INT32_MAX) x = -INFINITY;   // no more: the turns go on, as the warp's other rows may have some
                    if (in && (threadIdx.x & 15) == 0)
                        ((float2 *)((char *)a.workspace + ws.best))[at * top_k + count] =
                            make_float2(x, __int_as_float(word == INT32_MAX ? -1 : word));
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        if (n0 + col_of(j) == word) acc[i][j] = -INFINITY;
                }
                if (in && (threadIdx.x & 15) == 0)
                    ((RowStat *)((char *)a.workspace + ws.part))[at] = {top == -INFINITY ? top : base, sum, u, count};
            } else if (in && (threadIdx.x & 15) == 0)
                ((float2 *)((char *)a.workspace + ws.part))[(int64_t)row * ws.tiles + blockIdx.x] =
                    make_float2(top == -INFINITY ? top : base, sum);
        }
    }
}

// A warp a row: joins the tiles' (max, sum) pairs.
__global__ void __launch_bounds__(256) ce_join_kernel(LinearCeArgs a, CeWorkspace ws)
{
    const int lane = threadIdx.x & 31;
    const int row = (blockIdx.x * 256 + threadIdx.x) >> 5;
    if (row >= a.N) return;
    const float2 *p = (const float2 *)((const char *)a.workspace + ws.part) + (int64_t)row * ws.tiles;
    float top = -INFINITY;
    for (int i = lane; i < ws.tiles; i += 32) top = fmaxf(top, p[i].x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    const float base = isinf(top) ? 0.f : top;
    float sum = 0.f;
    for (int i = lane; i < ws.tiles; i += 32) sum += p[i].y * expf(p[i].x - base);
    sum = warp_sum(sum);
    if (lane == 0) {
        const bool keep = kept(a, row);
        const float lse = base + logf(sum);
        if (a.loss) a.loss[row] = keep ? lse - ((const float *)((const char *)a.workspace + ws.at))[row] : 0.f;
        if (a.lse) a.lse[row] = keep ? lse : 0.f;
    }
}

// dh (+)= G W over one piece; the last piece writes the gradient.
template <typename T>
__global__ void __launch_bounds__(kThreads, 2) ce_dh_kernel(LinearCeArgs a, CeWorkspace ws, int v0, int cols, int row0)
{
    const int m0 = row0 + blockIdx.y * kTile, n0 = blockIdx.x * kTile;
    const float *G = (const float *)((const char *)a.workspace + ws.g);
    float *sofar = (float *)((char *)a.workspace + ws.acc);
    const T *w = (const T *)a.w;
    float acc[8][8];
    tile_product<false, true>(
        [&](int m, int64_t k) { return m0 + m < a.N ? G[(int64_t)(m0 + m) * cols + k] : 0.f; },
        [&](int n, int64_t k) { return n0 + n < a.D ? to_f32(w[(v0 + k) * a.D + n0 + n]) : 0.f; }, cols, acc);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int row = m0 + row_of(i);
        if (row >= a.N) continue;
        const bool keep = kept(a, row);   // 0 times what W holds may be NaN
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int d = n0 + col_of(j);
            if (d >= a.D) continue;
            const int64_t at = (int64_t)row * a.D + d;
            const float s = v0 > 0 ? sofar[at] + acc[i][j] : acc[i][j];
            if (v0 + cols < a.V) sofar[at] = s;
            else ((T *)a.dh)[at] = from_f32<T>(keep ? s : 0.f);
        }
    }
}

// dW of one piece: G^T h over the kept rows.
template <typename T>
__global__ void __launch_bounds__(kThreads, 2) ce_dw_kernel(LinearCeArgs a, CeWorkspace ws, int v0, int cols, int row0)
{
    const int m0 = row0 + blockIdx.y * kTile, n0 = blockIdx.x * kTile;
    const float *G = (const float *)((const char *)a.workspace + ws.g);
    const T *h = (const T *)a.h;
    float acc[8][8];
    tile_product<true, true>(
        [&](int m, int64_t k) { return m0 + m < cols ? G[k * cols + m0 + m] : 0.f; },
        [&](int n, int64_t k) { return n0 + n < a.D && kept(a, (int)k) ? to_f32(h[k * a.D + n0 + n]) : 0.f; }, a.N, acc);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int v = m0 + row_of(i);
        if (v >= cols) continue;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int d = n0 + col_of(j);
            if (d < a.D) ((T *)a.dw)[(int64_t)(v0 + v) * a.D + d] = from_f32<T>(acc[i][j]);
        }
    }
}

// launch(grid, row0) over the tiles of rows x columns: a grid's second index ends at 65535, so more rows of tiles than that
// are several launches.
template <class Launch>
void over_tiles(int rows, int columns, Launch launch)
{
    constexpr int kMost = 65535;
    const int down = ceil_div(rows, kTile);
    for (int first = 0; first < down; first += kMost)
        launch(dim3(ceil_div(columns, kTile), down - first < kMost ? down - first : kMost), first * kTile);
}

template <typename T>
cudaError_t fwd(const LinearCeArgs &a, cudaStream_t st, const LogProbs *out)
{
    if (out) {
        const CeWorkspace ws = layout(a.N, a.D, a.V, false, out->top_k);
        over_tiles(a.N, a.V, [&](dim3 grid, int row0) {
            ce_logits_kernel<T, kStats><<<grid, kThreads, 0, st>>>(a, ws, 0, a.V, row0, LogProbsGrad(), out->top_k);
        });
        const char *w = (const char *)a.workspace;
        const LogProbParts p = {(const RowStat *)(w + ws.part), (const float2 *)(w + ws.best), (const float *)(w + ws.at),
                                a.targets, nullptr, a.N, a.V, out->top_k, ws.tiles, PartOrder()};
        const int blocks = ceil_div(a.N, 8);
        if (out->top_k == 0) logp_join_kernel<0><<<blocks, 256, 0, st>>>(p, *out);
        else if (out->top_k <= 8) logp_join_kernel<8><<<blocks, 256, 0, st>>>(p, *out);
        else logp_join_kernel<kMostTop><<<blocks, 256, 0, st>>>(p, *out);
        return cudaGetLastError();
    }
    const CeWorkspace ws = layout(a.N, a.D, a.V, false);
    over_tiles(a.N, a.V, [&](dim3 grid, int row0) {
        ce_logits_kernel<T, kLoss><<<grid, kThreads, 0, st>>>(a, ws, 0, a.V, row0, LogProbsGrad(), 0);
    });
    ce_join_kernel<<<ceil_div(a.N, 8), 256, 0, st>>>(a, ws);
    return cudaGetLastError();
}

template <typename T>
cudaError_t bwd(const LinearCeArgs &a, cudaStream_t st, LogProbsGrad grad)
{
    const CeWorkspace ws = layout(a.N, a.D, a.V, true);
    for (int v0 = 0; v0 < a.V; v0 += ws.piece) {
        const int cols = a.V - v0 < ws.piece ? a.V - v0 : ws.piece;
        over_tiles(a.N, cols, [&](dim3 grid, int row0) {
            (grad.dentropy ? ce_logits_kernel<T, kBackEnt> : ce_logits_kernel<T, kBack>)
                <<<grid, kThreads, 0, st>>>(a, ws, v0, cols, row0, grad, 0);
        });
        if (a.dh)
            over_tiles(a.N, a.D, [&](dim3 grid, int row0) {
                ce_dh_kernel<T><<<grid, kThreads, 0, st>>>(a, ws, v0, cols, row0);
            });
        if (a.dw)
            over_tiles(cols, a.D, [&](dim3 grid, int row0) {
                ce_dw_kernel<T><<<grid, kThreads, 0, st>>>(a, ws, v0, cols, row0);
            });
    }
    return cudaGetLastError();
}

}  // namespace

size_t linear_ce_workspace_bytes(int N, int D, int V, int dt, bool backward, int top)
{
    if (linear_ce_tc_supported(dt, D)) return linear_ce_tc_workspace_bytes(N, D, V, backward, top);
    return 256 + layout(N, D, V, backward, top).total;
}

cudaError_t launch_linear_ce_fwd(const LinearCeArgs &a0, cudaStream_t st, const LogProbs *out)
{
    if (linear_ce_tc_supported(a0.dt, a0.D)) return launch_linear_ce_tc_fwd(a0, st, out);
    LinearCeArgs a = a0;
    a.workspace = (char *)a0.workspace + 256;
    return a.dt ? fwd<__nv_bfloat16>(a, st, out) : fwd<float>(a, st, out);
}

cudaError_t launch_linear_ce_bwd(const LinearCeArgs &a0, cudaStream_t st, LogProbsGrad grad)
{
    if (linear_ce_tc_supported(a0.dt, a0.D)) return launch_linear_ce_tc_bwd(a0, st, grad);
    LinearCeArgs a = a0;
    a.workspace = (char *)a0.workspace + 256;
    return a.dt ? bwd<__nv_bfloat16>(a, st, grad) : bwd<float>(a, st, grad);
}

}  // namespace gdn
