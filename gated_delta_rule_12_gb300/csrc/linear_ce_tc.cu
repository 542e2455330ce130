// linear_ce_tc.cu -- the linear cross entropy's products on the tensor cores (bf16, D a multiple of 8).
//
// One persistent kernel form serves the three products, each over 256 x 256 tiles of a pair of CTAs:
//   logits   [h | w]     A = h  (K = D contiguous),     B = w (K contiguous):    a row's (max, sum) per tile
//   E        same operands, recomputed for one piece of the vocabulary:          E = softmax - onehot, bf16
//            (with an entropy's gradient: the gradient of the logits in units of the row's weight, below)
//   gradients            dW: A = E^T, B = dloss h (both with K = tokens as rows),  dW of the piece
//                        dh: A = E (K = words contiguous), B = w (K as rows),    fp32 sums over the pieces
// Tile: tcgen05.mma cta_group::2, M = 256 (128 rows a CTA), N = 256, K = 16 a step; a CTA holds 128 rows of A and
// 128 columns of B of each 64-deep stage (32 KB, six stages), its 128 x 256 fp32 accumulator in tensor memory, two of
// them, so that one tile's epilogue runs under the next one's products.  A pair reads half of B per CTA, which
// brings shared-memory traffic under the 128 B a clock that one-CTA tiles of this size exceed.
// Roles: warp 0 issues the TMA loads of its CTA, warp 1 of the even CTA the MMAs, warps 2-5 the epilogue (a thread a
// row; 32 tensor-memory lanes a warp).  Eight epilogue warps, half of the columns each, measured slower (255 tokens,
// 50257 words: 35 us against 31), and so did tiles of fewer columns where they fill the last round of pairs better
// (225 tiles of 224 columns instead of 197 of 256: 30.0 us against 29.6; 8192 x 2048 x 32768 with 128: 918 against 547).
//
// Precision: operands are bf16, sums fp32.  E is rounded to bf16 (relative 2^-8, independent from entry to entry, as
// exact as the inputs that it meets).  It is kept free of dloss: a target's entry is mostly close to -1, where bf16 is
// exact, while -dloss rounds, for a mean over the tokens, to one and the same relative error of up to 2^-8 in every
// row (8192 tokens, 65536 words: error of both gradients 3.3e-3 with dloss inside, against 1.7e-3 of the result's own
// rounding).  dh takes dloss in fp32 at its end.  dW takes it through its other operand, h dloss / s with s = max
// |dloss| over the kept rows, which is h itself where all rows weigh the same, and multiplies by s in fp32 at its end.
// Rows of unequal weights round there once more: weights uniform in (0, 1) or log-normal leave dW's error at 2.3e-3.
// The exponentials are the hardware's (2 ulp and the argument's rounding) and the products' sums are the tensor cores': the
// loss is off by 3.1e-7 of its size (255 x 1024 x 50257) and 7.0e-7 (8192 x 2048 x 32768), where fp32 products and expf
// leave 5e-8 and 7e-8.
//
// The log probabilities are the same products: their forward pass adds the entropy's sum to a row's statistics and keeps a
// row's best words (log_probs.cuh), their gradient is another E.  8192 x 2048 x 32768 0.50 ms without alternatives, 0.54 with
// five and 0.64 with twenty; 255 x 1024 x 50257 28, 46 (eight) and 88 us: a row's first tile costs the epilogue some 6 us (16
// with twenty), one word after another out of each of 32 rows, which only products of a few thousand terms cover.  Over short
// rows of h the epilogue is all that counts: 8192 x 256 x 32768 0.22 ms without alternatives, 0.39 with five, 0.56 with twenty,
// where the products take 0.072.
//
// Bound by the tensor cores, or by reading w where tokens are few.  Measured on the device: loss of 8192 x 2048 x 32768
// 0.54 ms (2.0 PFLOP/s), gradient with 65536 words 3.6 ms (1.83 PFLOP/s); both run into the power limit when repeated
// (0.61 and 3.9 to 4.1 ms).  Loss of 255 x 1024 x 50257 29 us, half of the copy rate: three rounds of tiles and what
// surrounds them.
//
// Every wait on an mbarrier is bounded (1 s); a timeout records kDevErrTimeout in the workspace's error word, and the
// CTA's roles unwind to the common exit, where both CTAs meet before tensor memory is freed.  Most callers never see that
// word, so a CTA that gave up then writes NaN over all its tiles: the loss, or the rows and words that they reach, are NaN.
#include <stdint.h>
#include <string.h>

#include "common.cuh"
#include "kernels.h"
#include "log_probs.cuh"
#include "pair_mma.cuh"
#include "umma.cuh"

namespace gdn {
namespace {

using namespace umma;

constexpr int kTile = 256;                 // rows and columns of a pair's tile
constexpr int kHalf = 128;                 // a CTA's rows of A and of B
constexpr int kDepth = 64;                 // K of one stage: 128 B, the swizzle's width
constexpr int kStages = 6;
constexpr int kStageBytes = 2 * kHalf * kDepth * 2;
constexpr int kStore = 4096;               // a warp's store buffer: 32 rows of 128 B
constexpr int kEpilogueWarps = 4;
constexpr int kThreads = 64 + 32 * kEpilogueWarps;
constexpr int kSmem = 1024 + kStages * kStageBytes + kEpilogueWarps * kStore + 256;
constexpr uint64_t kWaitLimitNs = 1000000000ull;
constexpr int kPairs = 76;                 // CTA pairs the GPU holds at once (152 SMs)

// kStats: kLogits with what the entropy takes, and a row's best words; kProbEnt: kProb with the entropy's gradient.
enum { kLogits = 0, kProb = 1, kGrads = 2, kStats = 3, kProbEnt = 4 };

// What a row's gradient of the logits is kept free of: the cross entropy's dloss (sign 1), minus the gradient of a token's
// log probability (sign -1), or, with a gradient b of the entropy, |a|, and |b| where that is 2^20 times larger: a target's
// entry is close to 1 in units of |a|.  (In units of a power of two dW's other operand stays exact, but that entry's rounding
// is one and the same relative error of the whole row: a single token 3.9e-3 instead of 2.0e-3.)
struct RowWeights {
    const float *a, *b;
    float sign;
    __device__ __forceinline__ float operator()(int row) const
    {
        const float x = __ldg(a + row);
        if (!b) return sign * x;
        const float y = fabsf(__ldg(b + row));
        return fabsf(x) * 0x1p20f >= y ? fabsf(x) : y;   // (the smallest y has no multiple by 2^-20)
    }
};

// One product C[M, N] = A B^T over `kb` stages of K.
struct Product {
    int mt, nt;       // tiles
    int kb;           // 64-deep stages along K
    int slices;       // K is cut into this many tiles
    int b_row0;       // first row of B's array that K (or, for logits, N) starts at
};

struct CeParams {
    Product p[2];             // kGrads: dW, dh; else p[0]
    int tiles0, tiles;        // tiles of p[0]; of both
    int N, V, D;
    int v0, cols;             // the piece (kProb), the whole vocabulary (kLogits)
    int accumulate;           // kGrads: dh adds to the earlier pieces' sums
    int direct;               // kGrads: the only piece, dh in one slice: its tiles are the result
    const int32_t *targets;
    const float *lse_in, *entropy;
    RowWeights weight;
    const float *scale;       // kGrads: s
    float2 *part;             // kLogits: [tiles of 256 words][N]
    RowStat *stat;            // kStats: [parts as `order` has them]
    float2 *best;             // kStats: [the same][top], a logit and its word's bits
    PartOrder order;          // kStats
    unsigned *cut;            // kStats: [N], order_of() of a logit that the row's best words do not fall below; or null
    int top;
    float *at;                // kLogits, kStats: [N]
    unsigned *err;
    int clear_err;            // the call's first kernel
    void *out[2];             // kProb: E; kGrads: dW of the piece, dh or its slices
    int pitch;                // kProb: elements a row of E
    uint64_t limit_ns;        // of a wait
    int silent;               // the self-test: the pair whose loads never come, else -1
};

struct CeMaps {
    CUtensorMap a[2], b[2], out[2];
};

__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, volatile int *abort_flag, const CeParams &p)
{
    return wait_cluster(bar, parity, abort_flag, p.err, p.limit_ns);
}

// Which product, tile and K range a tile index stands for.
struct Tile {
    int which, m, n, s, k0, k1;
    int part;                 // kStats
};

template <int MODE>
__device__ __forceinline__ Tile tile_of(const CeParams &p, int t)
{
    Tile r = {};
    if (MODE == kStats) {
        if (p.order.at(t % p.order.pairs, t / p.order.pairs, r.m, r.n, r.part)) r.k1 = p.p[0].kb;   // else nothing to do
    } else if (MODE == kGrads) {
        r.which = t >= p.tiles0;
        const Product &q = p.p[r.which];
        int i = r.which ? t - p.tiles0 : t;
        r.n = i % q.nt;            // the neighbours share A's rows: E is read from memory once
        i /= q.nt;
        r.s = i % q.slices;
        r.m = i / q.slices;
        r.k0 = (int)((int64_t)q.kb * r.s / q.slices);
        r.k1 = (int)((int64_t)q.kb * (r.s + 1) / q.slices);
    } else {
        // groups of up to 32 row tiles, whose h stays in L2 while the vocabulary passes by
        const Product &q = p.p[0];
        const int group = t / (32 * q.nt), first = group * 32, rows = min(32, q.mt - first);
        const int i = t - group * 32 * q.nt;
        r.which = 0;
        r.m = first + i % rows;
        r.n = i / rows;
        r.s = 0;
        r.k0 = 0;
        r.k1 = q.kb;
    }
    return r;
}

// Where a row's part lies.
__device__ __forceinline__ int64_t part_of(const CeParams &p, int part, int row)
{
    return p.order.first(row) + part * p.order.step(row, p.N);
}

// NaN in this CTA's half of each of the pair's tiles.
template <int MODE>
__device__ __noinline__ void spoil(const CeParams &p, int pair, int pairs, int rank)
{
    for (int t = pair; t < p.tiles; t += pairs) {
        const Tile c = tile_of<MODE>(p, t);
        if (c.k0 >= c.k1) continue;
        const int row0 = c.m * kTile + rank * kHalf, col0 = c.n * kTile;
        const int rows = min(kHalf, (MODE == kGrads && c.which == 0 ? p.cols : p.N) - row0);
        const int cols = min(kTile, (MODE == kGrads ? p.D : p.cols) - col0);
        for (int i = threadIdx.x; i < rows * cols; i += kThreads) {
            const int64_t row = row0 + i / cols;
            const int col = col0 + i % cols;
            const float nan = __uint_as_float(0x7fffffffu);
            if (MODE == kLogits) {
                p.part[(int64_t)c.n * p.N + row] = make_float2(nan, nan);
            } else if (MODE == kStats) {
                p.stat[part_of(p, c.part, (int)row)] = {nan, nan, nan, 0};
            } else if (MODE == kProb || MODE == kProbEnt) {
                static_cast<unsigned short *>(p.out[0])[row * p.pitch + col] = 0x7fff;
            } else if (c.which == 0 || p.direct) {
                static_cast<unsigned short *>(p.out[c.which])[row * p.D + col] = 0x7fff;
            } else {
                static_cast<unsigned *>(p.out[1])[((int64_t)c.s * p.N + row) * p.D + col] = 0x7fffffffu;
            }
        }
    }
}

// K: the best words that a thread keeps in kStats, at least p.top.
template <int MODE, int K = 0>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
ce_tc_kernel(const __grid_constant__ CeMaps maps, const __grid_constant__ CeParams p)
{
    constexpr int kWarpStore = K ? 2 * kStore : kStore;   // K: 64 words of each of a warp's rows
    extern __shared__ unsigned char smem_raw[];
    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    const uint32_t stores = base + kStages * kStageBytes;
    const uint32_t bars = stores + kEpilogueWarps * kWarpStore;
    const uint32_t full = bars, empty = bars + 8 * kStages, acc_full = bars + 16 * kStages, acc_empty = acc_full + 16;
    const uint32_t tmem_slot = acc_empty + 16, abort_addr = tmem_slot + 4;
    unsigned char *gen = smem_raw + (base - smem_u32(smem_raw));
    volatile int *abort_flag = reinterpret_cast<volatile int *>(gen + (abort_addr - base));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();

    if (threadIdx.x == 32) {
        prefetch_tmap(&maps.a[0]);
        prefetch_tmap(&maps.b[0]);
        if (MODE == kGrads) { prefetch_tmap(&maps.a[1]); prefetch_tmap(&maps.b[1]); }
    }
    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(full + 8 * i, 1);
            mbar_init(empty + 8 * i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(acc_full + 8 * i, 1);
            mbar_init(acc_empty + 8 * i, 2 * kEpilogueWarps);   // of both CTAs
        }
        fence_mbar_init();
        *abort_flag = 0;
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;"
                     :: "r"(tmem_slot), "r"(512u) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    fence_before_sync();
    __syncthreads();
    cluster_sync();
    fence_after_sync();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(gen + (tmem_slot - base));
    // The next kernel of the stream may take the SMs as they fall free; this one touches memory once the last is done.
    start_next();
    wait_previous();
    if (threadIdx.x == 0 && blockIdx.x == 0 && p.clear_err) *p.err = kDevErrNone;   // a timeout comes a second later at the earliest

    const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
    if (warp == 0) {
        if (lane == 0) {
            uint32_t it = 0;
            bool ok = true;
            for (int t = pair == p.silent ? p.tiles : pair; t < p.tiles && ok; t += pairs) {
                const Tile c = tile_of<MODE>(p, t);
                const Product &q = p.p[c.which];
                const CUtensorMap *ma = &maps.a[c.which], *mb = &maps.b[c.which];
                const bool a_mn = MODE == kGrads && c.which == 0, b_mn = MODE == kGrads;
                const int m0 = c.m * kTile + (int)rank * kHalf, n0 = c.n * kTile + (int)rank * kHalf;
                for (int k = c.k0; k < c.k1; ++k, ++it) {
                    const uint32_t s = it % kStages, ph = (it / kStages) & 1;
                    if (!wait_bar(empty + 8 * s, ph ^ 1, abort_flag, p)) { ok = false; break; }
                    const uint32_t bar = map_to_rank(full + 8 * s, 0);
                    if (rank == 0) mbar_expect_tx(full + 8 * s, 2 * kStageBytes);
                    const uint32_t sa = base + s * kStageBytes, sb = sa + kStageBytes / 2;
                    if (a_mn) {
                        load_2d(sa, ma, m0, k * kDepth, bar);
                        load_2d(sa + 8192, ma, m0 + 64, k * kDepth, bar);
                    } else {
                        load_2d(sa, ma, k * kDepth, m0, bar);
                    }
                    if (b_mn) {
                        load_2d(sb, mb, n0, q.b_row0 + k * kDepth, bar);
                        load_2d(sb + 8192, mb, n0 + 64, q.b_row0 + k * kDepth, bar);
                    } else {
                        load_2d(sb, mb, k * kDepth, q.b_row0 + n0, bar);
                    }
                }
            }
            // no copy and no arrival may come after the CTA has left: the last fills of the stages are read first
            const uint32_t n = it < (uint32_t)kStages ? it : kStages;
            for (uint32_t j = it - n; j < it && ok; ++j)
                ok = wait_bar(empty + 8 * (j % kStages), (j / kStages) & 1, abort_flag, p);
            if (!ok) {   // given up: copies in flight get 10 ms to land
                const uint64_t t0 = globaltimer_ns();
                while (globaltimer_ns() - t0 < 10000000ull) __nanosleep(1000);
            }
        }
    } else if (warp == 1) {
        if (rank == 0 && lane == 0) {
            uint32_t it = 0, tiles = 0;
            bool ok = true;
            for (int t = pair; t < p.tiles && ok; t += pairs) {
                const Tile c = tile_of<MODE>(p, t);
                if (c.k0 >= c.k1) continue;
                const bool a_mn = MODE == kGrads && c.which == 0, b_mn = MODE == kGrads;
                const uint32_t idesc = idesc_bf16(kTile, kTile, a_mn, b_mn);
                const uint32_t buf = tiles & 1, use = tiles >> 1;
                ++tiles;
                if (!wait_bar(acc_empty + 8 * buf, (use & 1) ^ 1, abort_flag, p)) break;
                fence_after_sync();
                const uint32_t d = tmem + buf * 256;
                const uint32_t a_step = a_mn ? 2048 : 32, b_step = b_mn ? 2048 : 32;
                for (int k = c.k0; k < c.k1; ++k, ++it) {
                    const uint32_t s = it % kStages, ph = (it / kStages) & 1;
                    if (!wait_bar(full + 8 * s, ph, abort_flag, p)) { ok = false; break; }
                    fence_after_sync();
                    const uint32_t sa = base + s * kStageBytes, sb = sa + kStageBytes / 2;
#pragma unroll
                    for (uint32_t j = 0; j < kDepth / 16; ++j)
                        mma_pair(d, smem_desc(sa + j * a_step, 8192, 1024), smem_desc(sb + j * b_step, 8192, 1024),
                                 idesc, (k > c.k0 || j > 0) ? 1u : 0u);
                    commit_pair(empty + 8 * s);
                }
                if (ok) commit_pair(acc_full + 8 * buf);
            }
        }
    } else {
        const uint32_t quarter = warp & 3;                     // the 32 tensor-memory lanes a warp may read
        constexpr int chunks = kTile / 32;
        const uint32_t buf0 = stores + (warp - 2) * kWarpStore;
        const uint32_t leader_empty = map_to_rank(acc_empty, 0);
        uint32_t tiles = 0;
        float top = -INFINITY, sum = 0.f, u = 0.f;
        // kStats: what the pair has seen of these rows so far
        BestWords<K ? K : 1> best;
        float cut = -INFINITY;                         // words at or below it are not among the row's best
        bool begins = true;
        Tile next = tile_of<MODE>(p, pair);
        for (int t = pair; t < p.tiles; t += pairs) {
            const Tile c = next;
            if (t + pairs < p.tiles) next = tile_of<MODE>(p, t + pairs);
            if (c.k0 >= c.k1) continue;
            const uint32_t buf = tiles & 1, use = tiles >> 1;
            ++tiles;
            const int row0 = c.m * kTile + (int)rank * kHalf + (int)quarter * 32, row = row0 + lane;
            const int col0 = c.n * kTile;
            const bool in = row < p.N;
            int target = -1;
            float lse = 0.f, scale = 1.f;
            const bool direct = MODE == kGrads && c.which == 1 && p.direct;
            if ((MODE != kGrads || direct) && in) {
                target = __ldg(p.targets + row);
                if (MODE == kProb || MODE == kProbEnt) lse = __ldg(p.lse_in + row);
                if (direct) scale = p.weight(row);
            }
            float ca = 0.f, cb = 0.f, entropy = 0.f;   // kProbEnt: the gradients in units of the row's weight
            if (MODE == kProbEnt && in) {
                const float r = p.weight(row), unit = r != 0.f ? r : 1.f;   // the least weights have no reciprocal
                ca = __ldg(p.weight.a + row) / unit;
                cb = __ldg(p.weight.b + row) / unit;
                entropy = __ldg(p.entropy + row);
            }
            if (MODE == kGrads && c.which == 0) scale = __ldg(p.scale);
            auto told = [&] { return K && in && p.cut ? *(volatile const unsigned *)(p.cut + row) : 0u; };
            unsigned other = told();                   // what other tiles have found: words equal to it may be among the best
            const bool keep = (MODE == kGrads && !direct) || (target >= 0 && target < p.V);
            if (!__all_sync(0xffffffffu, wait_bar(acc_full + 8 * buf, use & 1, abort_flag, p))) break;
            fence_after_sync();
            const uint32_t src = tmem + buf * 256 + (quarter << 21);   // lane field: bits 16 and up
            if (begins) {
                top = -INFINITY;
                sum = u = 0.f;
                cut = -INFINITY;
                best = BestWords<K ? K : 1>();
            }
            const bool ends = MODE != kStats || t + pairs >= p.tiles || next.k0 >= next.k1 || next.m != c.m || next.part != c.part;
            begins = ends;
            if (K && other) cut = fmaxf(cut, below(other));
            const bool fresh = K && __any_sync(0xffffffffu, in && cut == -INFINITY);
            unsigned hot = 0u;                         // chunks with words above it
            float most[K ? 32 : 1];                    // fresh: the largest of every 32nd word
#pragma unroll
            for (int j = 0; j < (K ? 32 : 1); ++j) most[j] = -INFINITY;
#pragma unroll 1
            for (int ch = 0; ch < chunks; ++ch) {
                uint32_t r[32];
                tmem_ld32(src + ch * 32, r);
                tmem_wait_ld();
                if (!K && ch == chunks - 1) {   // the accumulator is in registers: the next tile but one may have it
                    fence_before_sync();
                    __syncwarp();
                    if (lane == 0) arrive_remote(leader_empty + 8 * buf);
                }
                const int c0 = col0 + ch * 32;   // within the piece for kProb
                if (MODE == kLogits || MODE == kStats) {
                    if (c0 + 32 > p.V) {
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            if (c0 + j >= p.V) r[j] = 0xff800000u;   // -inf: no such word
                    }
                    if ((unsigned)(target - c0) < 32u && target < p.V) {
                        float x = 0.f;
#pragma unroll
                        for (int j = 0; j < 32; ++j) x = (target - c0 == j) ? __uint_as_float(r[j]) : x;
                        p.at[row] = x;
                    }
                    float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                    for (int j = 0; j < 32; ++j) m4[j & 3] = fmaxf(m4[j & 3], __uint_as_float(r[j]));
                    const float here = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])), higher = fmaxf(top, here);
                    // the base keeps infinities and NaN in the sum instead of making them NaN by themselves
                    const float was = isinf(top) ? 0.f : top, now = isinf(higher) ? 0.f : higher;
                    if (top != -INFINITY) {
                        // words masked by the lowest number lie so far below that the distance times their sum is infinite
                        const float d = MODE == kStats ? fmaxf(was - now, -1e4f) : was - now, f = __expf(d);
                        if (MODE == kStats) u = f * fmaf(d, sum, u);
                        sum *= f;
                    }
                    top = higher;
                    float s4[4] = {0.f, 0.f, 0.f, 0.f}, u4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int j = 0; j < 32; ++j) {
                        const float d = __uint_as_float(r[j]) - now, e = __expf(d);
                        s4[j & 3] += e;
                        if (MODE == kStats) u4[j & 3] = fmaf(e, fmaxf(d, -1e4f), u4[j & 3]);   // 0 times -inf is 0 here
                    }
                    sum += (s4[0] + s4[1]) + (s4[2] + s4[3]);
                    if (MODE == kStats) u += (u4[0] + u4[1]) + (u4[2] + u4[3]);
                    if (K) {
                        hot |= (here > cut ? 1u : 0u) << ch;
                        if (fresh)
#pragma unroll
                            for (int j = 0; j < 32; ++j) most[K ? j : 0] = fmaxf(most[K ? j : 0], __uint_as_float(r[j]));
                    }
                } else {
                    // 128-byte rows of the warp's buffer: 64 bf16, two chunks of 32 columns, or 32 fp32
                    const bool fp32 = MODE == kGrads && c.which == 1 && !direct;
                    const int part = fp32 ? 0 : ch & 1;
                    if (part == 0) {   // the buffer is written again once the last store has read it
                        if (lane == 0) bulk_wait_read();
                        __syncwarp();
                    }
                    const uint32_t buf_s = buf0 + lane * 128;
                    if (fp32) {
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            st_shared16(buf_s + ((j ^ (lane & 7)) << 4), r[4 * j], r[4 * j + 1], r[4 * j + 2],
                                        r[4 * j + 3]);
                    } else {
                        if (MODE == kProb) {
                            const int hot = target - p.v0 - c0;
#pragma unroll
                            for (int j = 0; j < 32; ++j) {
                                const float e = __expf(__uint_as_float(r[j]) - lse);
                                r[j] = __float_as_uint(keep ? e - (j == hot ? 1.f : 0.f) : 0.f);
                            }
                        } else if (MODE == kProbEnt) {
                            const int hot = target - p.v0 - c0;
#pragma unroll
                            for (int j = 0; j < 32; ++j) {
                                const float z = __uint_as_float(r[j]) - lse, e = __expf(z);
                                const float g = e * fmaf(cb, fmaxf(z, -1e4f) + entropy, ca);   // 0 times -inf is 0 here
                                r[j] = __float_as_uint(keep ? (j == hot ? ca : 0.f) - g : 0.f);
                            }
                        } else {
#pragma unroll
                            for (int j = 0; j < 32; ++j) r[j] = __float_as_uint(keep ? __uint_as_float(r[j]) * scale : 0.f);
                        }
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            uint32_t w[4];
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                w[i] = pack_bf16(__uint_as_float(r[8 * j + 2 * i]), __uint_as_float(r[8 * j + 2 * i + 1]));
                            st_shared16(buf_s + (((4 * part + j) ^ (lane & 7)) << 4), w[0], w[1], w[2], w[3]);
                        }
                    }
                    if (fp32 || part == 1) {
                        fence_proxy_async();
                        __syncwarp();
                        if (lane == 0) {
                            const uint32_t from = buf0;
                            const int x = fp32 ? c0 : c0 - 32;
                            if (MODE == kProb || MODE == kProbEnt) {
                                if (x < p.cols && row0 < p.N) store_2d(&maps.out[0], from, x, row0);
                            } else if (c.which == 0) {
                                if (x < p.D && row0 < p.cols) store_2d(&maps.out[0], from, x, p.v0 + row0);
                            } else if (x < p.D && row0 < p.N) {
                                if (direct) store_2d(&maps.out[1], from, x, row0);
                                else if (p.accumulate) add_3d(&maps.out[1], from, x, row0, c.s);
                                else store_3d(&maps.out[1], from, x, row0, c.s);
                            }
                            bulk_commit();
                        }
                    }
                }
            }
            if (MODE == kLogits && in)
                p.part[(int64_t)c.n * p.N + row] = make_float2(top == -INFINITY ? top : (isinf(top) ? 0.f : top), sum);
            if constexpr (K > 0) {
                // The words that may be among the row's best.  p.top of the 32 maxima are as many words, so what is below the
                // least of those is not; this and what other tiles tell leaves some 1.2 p.top words of a row's first tile.
                if (__any_sync(0xffffffffu, in && hot)) {
                    if (fresh) {
                        sort32(most);
                        float least = most[0];
#pragma unroll
                        for (int j = 1; j < K; ++j) least = j < p.top ? most[j] : least;
                        if (in && least > -INFINITY) {
                            if (p.cut) atomicMax(p.cut + row, order_of(least));
                            cut = fmaxf(cut, below(order_of(least)));
                        }
                        other = told();
                        if (other) cut = fmaxf(cut, below(other));
                    }
#pragma unroll 1
                    for (int ch = 0; ch < chunks; ch += 2) {   // 64 words at a time
                        unsigned some[2];
#pragma unroll
                        for (int half = 0; half < 2; ++half) {
                            some[half] = 0u;
                            if (!__any_sync(0xffffffffu, in && (hot >> (ch + half) & 1u))) continue;
                            uint32_t r[32];
                            tmem_ld32(src + (ch + half) * 32, r);
                            tmem_wait_ld();
                            const int c0 = col0 + (ch + half) * 32;
#pragma unroll
                            for (int j = 0; j < 32; ++j) some[half] |= (__uint_as_float(r[j]) > cut && c0 + j < p.V ? 1u : 0u) << j;
                            if (!in) some[half] = 0u;
#pragma unroll
                            for (int j = 0; j < 8; ++j)
                                st_shared16(buf0 + half * kStore + lane * 128 + ((j ^ (lane & 7)) << 4), r[4 * j], r[4 * j + 1],
                                            r[4 * j + 2], r[4 * j + 3]);
                        }
                        // They come out one at a time, each lane its own: found by their bits, then read back from the warp's
                        // buffer, as registers have no variable index; the next one is on its way while one is inserted.
                        auto take = [&](float &x, int &word) {
                            const int half = some[0] ? 0 : 1;
                            const unsigned m = half ? some[1] : some[0];
                            if (!m) return false;
                            const int j = __ffs((int)m) - 1;
                            if (half) some[1] &= m - 1u;
                            else some[0] &= m - 1u;
                            asm volatile("ld.shared.f32 %0, [%1];"
                                         : "=f"(x) : "r"(buf0 + half * kStore + lane * 128 + (((j >> 2) ^ (lane & 7)) << 4) + (j & 3) * 4)
                                         : "memory");
                            word = col0 + (ch + half) * 32 + j;
                            return true;
                        };
                        float x = 0.f, x2 = 0.f;
                        int word = 0, word2 = 0;
                        bool have = take(x, word);
                        while (__any_sync(0xffffffffu, have)) {
                            bool more = false;
                            if (have) {
                                more = take(x2, word2);
                                best.add(x, word);
                            }
                            have = more;
                            x = x2;
                            word = word2;
                        }
                        cut = fmaxf(cut, best.value(p.top - 1));
                    }
                }
                fence_before_sync();
                __syncwarp();
                if (lane == 0) arrive_remote(leader_empty + 8 * buf);
            }
            if (MODE == kStats && in && ends) {
                const int64_t at = part_of(p, c.part, row);
                const int count = K ? best.count(p.top) : 0;
                p.stat[at] = {top == -INFINITY ? top : (isinf(top) ? 0.f : top), sum, u, count};
                if (K) {
#pragma unroll
                    for (int i = 0; i < K; ++i)
                        if (i < count) p.best[at * p.top + i] = make_float2(best.v[i], __int_as_float(best.id[i]));
                    if (p.cut && count == p.top) atomicMax(p.cut + row, order_of(best.value(p.top - 1)));
                }
            }
        }
        if (MODE != kLogits && MODE != kStats && lane == 0) bulk_wait_all();
    }
    __syncwarp();
    fence_before_sync();
    __syncthreads();
    cluster_sync();
    fence_after_sync();
    if (warp == 1)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" :: "r"(tmem), "r"(512u) : "memory");
    if (*abort_flag) spoil<MODE>(p, pair, pairs, (int)rank);
}

// Joins a row's (max, sum) pairs: 32 rows a block, each warp a share of the `words` pairs of each, first the largest maximum,
// then the sums in its units.
constexpr int kJoinWarps = 16;

__global__ void __launch_bounds__(32 * kJoinWarps) ce_tc_join_kernel(const CeParams p, int words, float *loss, float *lse_out)
{
    __shared__ float tops[kJoinWarps][32], sums[kJoinWarps][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int row = blockIdx.x * 32 + lane;
    wait_previous();
    const float2 *part = p.part + (row < p.N ? row : 0);
    float top = -INFINITY, sum = 0.f;
#pragma unroll 8
    for (int i = warp; i < words; i += kJoinWarps) top = fmaxf(top, part[(int64_t)i * p.N].x);
    tops[warp][lane] = top;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kJoinWarps; ++i) top = fmaxf(top, tops[i][lane]);
    const float base = isinf(top) ? 0.f : top;   // keeps infinities and NaN in the sum
#pragma unroll 8
    for (int i = warp; i < words; i += kJoinWarps) {
        const float2 v = part[(int64_t)i * p.N];
        sum += v.y * expf(v.x - base);
    }
    sums[warp][lane] = sum;
    __syncthreads();
    if (warp == 0 && row < p.N) {
        sum = 0.f;
#pragma unroll
        for (int i = 0; i < kJoinWarps; ++i) sum += sums[i][lane];
        const int t = p.targets[row];
        const bool keep = t >= 0 && t < p.V;
        const float lse = base + logf(sum);
        loss[row] = keep ? lse - p.at[row] : 0.f;
        if (lse_out) lse_out[row] = keep ? lse : 0.f;
    }
}

// s = max |dloss| over the kept rows, finite, and 1 where that is 0; the same in every thread of the block.
__device__ __forceinline__ float largest_weight(RowWeights weight, const int32_t *targets, int N, int V)
{
    __shared__ float sh[32];
    float m = 0.f;
    for (int i = threadIdx.x; i < N; i += blockDim.x) {
        const int t = __ldg(targets + i);
        if (t >= 0 && t < V) m = fmaxf(m, fabsf(weight(i)));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = m;
    __syncthreads();
    m = 0.f;
    for (int i = 0; i < (int)blockDim.x / 32; ++i) m = fmaxf(m, sh[i]);
    return m > 0.f ? fminf(m, 3.402823466e38f) : 1.f;
}

__global__ void __launch_bounds__(1024) ce_scale_kernel(RowWeights weight, const int32_t *targets, int N, int V,
                                                        float *scale)
{
    const float s = largest_weight(weight, targets, N, V);
    if (threadIdx.x == 0) *scale = s;
}

__device__ __forceinline__ uint32_t scale_bf16x2(uint32_t v, float f)
{
    return pack_bf16(__uint_as_float(v << 16) * f, __uint_as_float(v & 0xffff0000u) * f);
}

// h dloss / s, the ignored rows zeroed: a zero of E times what such a row holds could be NaN.  OWN: every block finds
// s by itself, which is quicker than a launch before this one up to kOwnScale tokens.
constexpr int kOwnScale = 4096;

template <bool OWN>
__global__ void __launch_bounds__(256) ce_weighted_rows_kernel(const uint4 *h, uint4 *out, const int32_t *targets,
                                                               RowWeights weight, float *scale, int N, int D8, int V)
{
    const float s = OWN ? largest_weight(weight, targets, N, V) : *scale;
    if (OWN && blockIdx.x == 0 && threadIdx.x == 0) *scale = s;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < (int64_t)N * D8; i += (int64_t)gridDim.x * 256) {
        const int row = (int)(i / D8), t = __ldg(targets + row);
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        if (t >= 0 && t < V) {
            const float f = weight(row) / s;
            v = h[i];
            v = make_uint4(scale_bf16x2(v.x, f), scale_bf16x2(v.y, f), scale_bf16x2(v.z, f), scale_bf16x2(v.w, f));
        }
        out[i] = v;
    }
}

// dh = dloss times the sum of its slices, in order, rounded; 0 in the ignored rows.
__global__ void __launch_bounds__(256) ce_dh_finish_kernel(const float4 *acc, uint2 *dh, const int32_t *targets,
                                                           RowWeights weight, int N, int D4, int V, int slices)
{
    const int64_t n = (int64_t)N * D4;
    wait_previous();
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
        const int row = (int)(i / D4), t = __ldg(targets + row);
        const float f = weight(row);
        float4 s = acc[i];
        for (int j = 1; j < slices; ++j) {
            const float4 v = acc[i + j * n];
            s.x += v.x; s.y += v.y; s.z += v.z; s.w += v.w;
        }
        dh[i] = (t >= 0 && t < V) ? make_uint2(pack_bf16(s.x * f, s.y * f), pack_bf16(s.z * f, s.w * f))
                                  : make_uint2(0u, 0u);
    }
}

// [rows, cols] (and slices of them) with `pitch` elements a row; 128-B swizzled boxes of box_rows x 128 B.
bool make_map(CUtensorMap *m, const void *base, int cols, int rows, int64_t pitch, int box_rows, bool fp32 = false,
              int slices = 0)
{
    auto fn = encode_fn();
    if (!fn) return false;
    const int size = fp32 ? 4 : 2;
    cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)slices};
    cuuint64_t strides[2] = {(cuuint64_t)pitch * size, (cuuint64_t)pitch * rows * size};
    cuuint32_t box[3] = {(cuuint32_t)(128 / size), (cuuint32_t)box_rows, 1};
    cuuint32_t es[3] = {1, 1, 1};
    return fn(m, fp32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, slices ? 3 : 2,
              const_cast<void *>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

PartOrder part_order(int N, int V)
{
    const int mt = ceil_div(N > 0 ? N : 1, kTile), nt = ceil_div(V, kTile);
    return PartOrder::make(mt, nt, (int64_t)mt * nt < kPairs ? mt * nt : kPairs);
}

struct TcWorkspace {
    size_t part, at;          // forward: a row's statistics of each tile of words, log probabilities of each part; [N]
    size_t best, cut;         // log probabilities, forward: the rows' parts' best words (PartOrder), [N]
    // backward: E of a piece [N][piece], h dloss / s of the kept rows [N][D], dh's slices [.][N][D], s
    size_t e, hk, acc, scale;
    size_t total;
    int piece, slices;
    bool direct;              // one piece, one slice: dh needs no sums
};

// top: the best words of a log-probability call, -1 for the cross entropy
TcWorkspace tc_layout(int N, int D, int V, bool backward, int top = -1)
{
    TcWorkspace w = {};
    size_t off = 256;
    if (!backward) {
        const size_t parts = top < 0 ? (size_t)N * ceil_div(V, kTile) : (size_t)part_order(N, V).total(N);
        w.part = off; off = align256(off + parts * (top < 0 ? sizeof(float2) : sizeof(RowStat)));
        w.at = off;   off = align256(off + (size_t)N * 4);
        w.best = off; off = align256(off + (top > 0 ? parts * top * sizeof(float2) : 0));
        w.cut = off;  off = align256(off + (top > 0 ? (size_t)N * 4 : 0));
    } else {
        // pieces of equal size whose E takes up to 128 MB (8192 x 2048 x 65536: 32 MB 4.39 ms, 64 MB 3.99, 128 MB 3.67,
        // 512 MB 3.55)
        const int tiles = ceil_div(V, kTile);
        const int64_t fit = ((int64_t)64 << 20) / (N > 0 ? N : 1) / kTile;
        const int most = (int)(fit < 1 ? 1 : fit > tiles ? tiles : fit);
        const int per = ceil_div(tiles, ceil_div(tiles, most));
        w.piece = per * kTile;
        // dh has N D / 65536 tiles, each as long as the piece: few of them are cut along the piece
        const int dh_tiles = ceil_div(N > 0 ? N : 1, kTile) * ceil_div(D, kTile);
        int s = ceil_div(2 * kPairs, dh_tiles);
        if (s > 32) s = 32;
        if (s > per) s = per;      // four stages a slice at least
        if (per <= 4) s = 1;       // up to 1024 words in all: short enough, and no slices to join
        w.slices = s < 1 ? 1 : s;
        w.direct = w.slices == 1 && w.piece >= V;
        w.e = off;   off = align256(off + (size_t)N * w.piece * 2);
        w.hk = off;  off = align256(off + (size_t)N * D * 2);
        w.acc = off; off = align256(off + (w.direct ? 0 : (size_t)w.slices * N * D * 4));
        w.scale = off; off += 256;
    }
    w.total = off;
    return w;
}

template <int MODE, int K = 0>
cudaError_t launch(const CeMaps &maps, CeParams p, cudaStream_t st, const CeStall &stall)
{
    p.silent = stall.step == MODE ? 0 : -1;
    p.limit_ns = stall.step == MODE ? stall.limit_ns : kWaitLimitNs;
    constexpr int smem = kSmem + (K ? kEpilogueWarps * kStore : 0);
    const cudaError_t e = cudaFuncSetAttribute(ce_tc_kernel<MODE, K>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    const int pairs = p.tiles < kPairs ? p.tiles : kPairs;
    return launch_early(ce_tc_kernel<MODE, K>, 2 * pairs, kThreads, smem, st, maps, p);
}

unsigned grid_for(int64_t items)
{
    const int64_t b = (items + 255) / 256;
    return (unsigned)(b < 152 * 8 ? (b > 0 ? b : 1) : 152 * 8);
}

}  // namespace

// A tile's logits take D / 64 stages one after another, 0.26 us each where a pair is alone: 69 ms at 2^24, but the second
// after which the epilogue's wait gives up before 2^28.
bool linear_ce_tc_supported(int dt, int D) { return dt == 1 && D % 8 == 0 && D <= 1 << 24; }

size_t linear_ce_tc_workspace_bytes(int N, int D, int V, bool backward, int top)
{
    return tc_layout(N, D, V, backward, top).total;
}

template <int K>
static cudaError_t run_stats(const CeMaps &maps, const CeParams &p, const LogProbs &out, cudaStream_t st, const CeStall &stall)
{
    const cudaError_t e = launch<kStats, K>(maps, p, st, stall);
    if (e != cudaSuccess) return e;
    const LogProbParts parts = {p.stat, p.best, p.at, p.targets, p.cut, p.N, p.V, p.top, 0, p.order};
    return launch_early(logp_join_kernel<K>, ceil_div(p.N, 8), 256, 0, st, parts, out);
}

cudaError_t launch_linear_ce_tc_fwd(const LinearCeArgs &a, cudaStream_t st, const LogProbs *out, CeStall stall)
{
    const TcWorkspace ws = tc_layout(a.N, a.D, a.V, false, out ? out->top_k : -1);
    char *w = (char *)a.workspace;
    CeMaps maps;
    memset(&maps, 0, sizeof(maps));
    CeParams p = {};
    if (!make_map(&maps.a[0], a.h, a.D, a.N, a.D, kHalf) || !make_map(&maps.b[0], a.w, a.D, a.V, a.D, kHalf))
        return cudaErrorInvalidValue;
    p.p[0] = {ceil_div(a.N, kTile), ceil_div(a.V, kTile), ceil_div(a.D, kDepth), 1, 0};
    p.tiles0 = p.tiles = p.p[0].mt * p.p[0].nt;
    p.N = a.N; p.V = a.V; p.D = a.D; p.cols = a.V;
    p.targets = a.targets;
    p.part = (float2 *)(w + ws.part);
    p.at = (float *)(w + ws.at);
    p.err = (unsigned *)w;
    p.clear_err = 1;
    if (out) {
        p.stat = (RowStat *)(w + ws.part);
        p.best = (float2 *)(w + ws.best);
        p.top = out->top_k;
        p.order = part_order(a.N, a.V);
        p.tiles0 = p.tiles = p.order.pairs * p.order.rounds();
        // Tiles tell later ones of their rows what need not be kept, where there are rounds enough of them to tell: clearing
        // the words is a launch more (255 x 1024 x 50257, three rounds, top 8: 48.7 us without, 52.6 with; 8192 x 2048 x
        // 32768, top 5: 587 us without, 541 with; top 20: 937 and 703; 32 words at a time then).
        if (p.top > 0 && p.tiles > 4 * kPairs) {
            p.cut = (unsigned *)(w + ws.cut);
            const cudaError_t e = cudaMemsetAsync(p.cut, 0, (size_t)a.N * 4, st);
            if (e != cudaSuccess) return e;
        }
        return p.top == 0 ? run_stats<0>(maps, p, *out, st, stall)
               : p.top <= 8 ? run_stats<8>(maps, p, *out, st, stall) : run_stats<kMostTop>(maps, p, *out, st, stall);
    }
    const cudaError_t e = launch<kLogits>(maps, p, st, stall);
    if (e != cudaSuccess) return e;
    return launch_early(ce_tc_join_kernel, ceil_div(a.N, 32), 32 * kJoinWarps, 0, st, p, p.p[0].nt, a.loss, a.lse);
}

cudaError_t launch_linear_ce_tc_bwd(const LinearCeArgs &a, cudaStream_t st, LogProbsGrad grad, CeStall stall)
{
    const TcWorkspace ws = tc_layout(a.N, a.D, a.V, true);
    char *w = (char *)a.workspace;
    const int mt = ceil_div(a.N, kTile), dt = ceil_div(a.D, kTile);
    CeParams p = {};
    p.N = a.N; p.V = a.V; p.D = a.D;
    p.targets = a.targets; p.lse_in = a.lse_in; p.entropy = grad.entropy;
    p.weight = {a.dloss, grad.dentropy, grad.sign};
    p.direct = ws.direct;
    p.scale = (float *)(w + ws.scale);
    p.err = (unsigned *)w;
    if (a.dw) {
        const bool own = a.N <= kOwnScale;
        if (!own) ce_scale_kernel<<<1, 1024, 0, st>>>(p.weight, a.targets, a.N, a.V, (float *)(w + ws.scale));
        (own ? ce_weighted_rows_kernel<true> : ce_weighted_rows_kernel<false>)
            <<<grid_for((int64_t)a.N * a.D / 8), 256, 0, st>>>((const uint4 *)a.h, (uint4 *)(w + ws.hk), a.targets,
                                                               p.weight, (float *)(w + ws.scale), a.N, a.D / 8, a.V);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    CeMaps mg, md;
    memset(&mg, 0, sizeof(mg));
    memset(&md, 0, sizeof(md));
    bool ok = make_map(&mg.a[0], a.h, a.D, a.N, a.D, kHalf) && make_map(&mg.b[0], a.w, a.D, a.V, a.D, kHalf) &&
              make_map(&md.b[0], w + ws.hk, a.D, a.N, a.D, kDepth) && make_map(&md.b[1], a.w, a.D, a.V, a.D, kDepth) &&
              (!a.dh || (ws.direct ? make_map(&md.out[1], a.dh, a.D, a.N, a.D, 32)
                                   : make_map(&md.out[1], w + ws.acc, a.D, a.N, a.D, 32, true, ws.slices)));
    if (a.dw) ok = ok && make_map(&md.out[0], a.dw, a.D, a.V, a.D, 32);
    if (!ok) return cudaErrorInvalidValue;
    for (int v0 = 0; v0 < a.V; v0 += ws.piece) {
        const int cols = a.V - v0 < ws.piece ? a.V - v0 : ws.piece;
        if (v0 == 0 || cols < ws.piece) {
            ok = make_map(&mg.out[0], w + ws.e, cols, a.N, ws.piece, 32) &&
                 make_map(&md.a[0], w + ws.e, cols, a.N, ws.piece, kDepth) &&
                 make_map(&md.a[1], w + ws.e, cols, a.N, ws.piece, kHalf);
            if (!ok) return cudaErrorInvalidValue;
        }
        p.v0 = v0; p.cols = cols;
        p.clear_err = v0 == 0;
        p.p[0] = {mt, ceil_div(cols, kTile), ceil_div(a.D, kDepth), 1, v0};
        p.tiles0 = p.tiles = mt * p.p[0].nt;
        p.out[0] = w + ws.e;
        p.pitch = ws.piece;
        cudaError_t e = grad.dentropy ? launch<kProbEnt>(mg, p, st, stall) : launch<kProb>(mg, p, st, stall);
        if (e != cudaSuccess) return e;
        p.p[0] = {ceil_div(cols, kTile), dt, ceil_div(a.N, kDepth), 1, 0};
        p.p[1] = {mt, dt, ceil_div(cols, kDepth), ws.slices, v0};
        p.tiles0 = a.dw ? p.p[0].mt * dt : 0;
        p.tiles = p.tiles0 + (a.dh ? mt * dt * ws.slices : 0);
        p.accumulate = v0 > 0;
        p.out[0] = a.dw ? (char *)a.dw + (int64_t)v0 * a.D * 2 : nullptr;
        p.out[1] = ws.direct ? a.dh : w + ws.acc;
        p.clear_err = 0;
        e = launch<kGrads>(md, p, st, stall);
        if (e != cudaSuccess) return e;
    }
    if (!a.dh || ws.direct) return cudaSuccess;
    return launch_early(ce_dh_finish_kernel, grid_for((int64_t)a.N * a.D / 4), 256, 0, st, (const float4 *)(w + ws.acc),
                        (uint2 *)a.dh, a.targets, p.weight, a.N, a.D / 4, a.V, ws.slices);
}

}  // namespace gdn
