// fp8_linear_tc.cu -- the product of 8-bit operands with scales on the tensor cores (K a multiple of 16):
//     out_mn = sum_b xs_mb ws_{n / 128, b} sum_{k in block b} x_mk w_nk
// tcgen05.mma kind::f8f6f4 multiplies one block of 128 along K into tensor memory; the epilogue's warps read it back, times
// the block's two scales, into fp32 sums in registers while the next block is multiplied into the other half.  (The
// instructions that take scales themselves know powers of two only.)  Sums are rounded once, to bf16.
//
// Two kernels:
//   pair_kernel   many tokens: 256 tokens x 256 words a pair of CTAs (cta_group::2, each holds 128 rows of both operands,
//                 five stages of 32 KB); persistent, one pair's tile after another.  Eight epilogue warps, a thread 128
//                 sums of its token.
//                 Results go to memory by TMA, rows that it cannot address (words no multiple of 8) by plain stores.
//   few_kernel    few tokens: the words are the rows of the tile (128), 16 to 128 tokens its columns, so the weights'
//                 bytes, which such a call is bound by, take the whole width.  A cluster of up to eight CTAs shares a
//                 tile's K; their partial sums meet in shared memory and are added in the CTAs' order.
//
// Bound, for many tokens, by the chain from a block's multiplication over its reading back to the next multiplication into
// the same half of tensor memory, across both CTAs: 910 cycles a block, 470 of them multiplying (8192 x 2048 x 6144: 91 us on
// the device, 2.26 PFLOP/s, tensor pipe 53 %).  Measured on it: epilogue arrivals that release to the cluster instead of
// relaxed ones 221 us (the release waits for the scale loads in flight); waits with a suspend hint 95.6; scales one block
// ahead 91.5; sixteen epilogue warps 98 to 104, also with registers moved to them; 128 words a multiplication in four quarters
// of tensor memory 132 (109 with 256 there); 160 words and three accumulators 129; one forwarded arrival of the peer instead of
// eight 94; multiplications of a CTA's own with half of the words multicast to it 95.  For few tokens by latency: one token takes
// 5.2 us where its weights' bytes take 1.9.
//
// Every wait on an mbarrier is bounded (1 s); a timeout records kDevErrTimeout in the workspace's error word and leaves NaN
// in the tiles that it reaches.
#include <stdint.h>
#include <string.h>

#include "common.cuh"
#include "kernels.h"
#include "pair_mma.cuh"
#include "pairs.cuh"
#include "umma.cuh"

namespace gdn {
namespace {

using namespace umma;

constexpr int kDepth = kFp8Block;          // K of a stage: 128 B, the swizzle's width
constexpr uint64_t kWaitLimitNs = 1000000000ull;
constexpr int kPairs = 76;                 // CTA pairs the GPU holds at once (152 SMs)
constexpr unsigned short kNaN = 0x7fff;    // bf16

struct Fp8Params {
    int M, N, K;
    int mt, nt, kb;           // tiles; blocks along K
    int stages, splits;       // few_kernel
    const float *xs, *ws;
    __nv_bfloat16 *out;
    unsigned *err;
    uint64_t limit_ns;        // of a wait
    int silent;               // the self-test: the pair or CTA whose loads never come, else -1
};

struct Fp8Maps {
    CUtensorMap x, w, out;
};

// kind::f8f6f4 with e4m3 A and B (format code 0), both K-major, fp32 accumulate
__host__ __device__ constexpr uint32_t idesc_e4m3(int M, int N)
{
    return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

__device__ __forceinline__ void mma_fp8_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}\n"
        :: "r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate) : "memory");
}

__device__ __forceinline__ void mma_fp8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}\n"
        :: "r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate) : "memory");
}

// These kernels' barriers order tensor memory, by tcgen05 fences, and what the asynchronous proxy wrote, so their waits
// and arrivals need no wider ordering: a release to the cluster waits for the warp's loads in flight, GPU-wide latency on
// the chain of every block.
__device__ __forceinline__ bool wait_here(uint32_t bar, uint32_t parity, volatile int *abort_flag, const Fp8Params &p)
{
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = globaltimer_ns();
    for (;;) {
        for (int i = 0; i < 64; ++i)
            if (mbar_try_wait(bar, parity)) return true;
        if (*abort_flag) return false;
        if (globaltimer_ns() - t0 > p.limit_ns) {
            *abort_flag = 1;
            atomicExch(p.err, kDevErrTimeout);
            return false;
        }
    }
}

__device__ __forceinline__ void arrive_remote_relaxed(uint32_t bar)
{
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" :: "r"(bar) : "memory");
}

__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap *map, int x, int y, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];"
        :: "r"(dst), "l"(map), "r"(x), "r"(y), "r"(bar) : "memory");
}

// Waits for the loads from tensor memory, of which `r` is the last: nothing that uses it may come before.
__device__ __forceinline__ void wait_ld(uint32_t (&r)[32])
{
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
                   "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]),
                   "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]),
                   "+r"(r[30]), "+r"(r[31]) :: "memory");
}

__device__ __forceinline__ void wait_ld(uint32_t (&r)[16])
{
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
                 :: "memory");
}

__device__ __forceinline__ Pair pair_of(uint32_t lo, uint32_t hi) { return pair(__uint_as_float(lo), __uint_as_float(hi)); }

// ---------------------------------------------------------------------------
// many tokens
// ---------------------------------------------------------------------------

constexpr int kTile = 256, kHalf = 128;
constexpr int kStages = 5, kStageBytes = 2 * kHalf * kDepth;
constexpr int kStore = 8192;               // a warp's results: two boxes of 32 rows x 64 bf16
constexpr int kEpilogueWarps = 8;
constexpr int kPairThreads = 64 + 32 * kEpilogueWarps;
constexpr int kPairSmem = 1024 + kStages * kStageBytes + kEpilogueWarps * kStore + 256;

// groups of up to 32 row tiles, whose x stays in L2 while the words pass by
__device__ __forceinline__ void pair_tile(const Fp8Params &p, int t, int &m, int &n)
{
    const int group = t / (32 * p.nt), first = group * 32, rows = min(32, p.mt - first), i = t - group * 32 * p.nt;
    m = first + i % rows;
    n = i / rows;
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPairThreads, 1)
pair_kernel(const __grid_constant__ Fp8Maps maps, const __grid_constant__ Fp8Params p)
{
    extern __shared__ unsigned char smem_raw[];
    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    const uint32_t stores = base + kStages * kStageBytes;
    const uint32_t bars = stores + kEpilogueWarps * kStore;
    const uint32_t full = bars, empty = bars + 8 * kStages, acc_full = bars + 16 * kStages, acc_empty = acc_full + 16;
    const uint32_t tmem_slot = acc_empty + 16, abort_addr = tmem_slot + 4;
    unsigned char *gen = smem_raw + (base - smem_u32(smem_raw));
    volatile int *abort_flag = reinterpret_cast<volatile int *>(gen + (abort_addr - base));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    auto wait = [&](uint32_t bar, uint32_t parity) { return wait_here(bar, parity, abort_flag, p); };

    if (threadIdx.x == 32) {
        prefetch_tmap(&maps.x);
        prefetch_tmap(&maps.w);
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
    if (threadIdx.x == 0 && blockIdx.x == 0) *p.err = kDevErrNone;   // a timeout comes a second later at the earliest

    const int pair_id = blockIdx.x >> 1, pairs = gridDim.x >> 1, tiles = p.mt * p.nt;
    if (warp == 0) {
        if (lane == 0) {
            uint32_t it = 0;
            bool ok = true;
            for (int t = pair_id == p.silent ? tiles : pair_id; t < tiles && ok; t += pairs) {
                int m, n;
                pair_tile(p, t, m, n);
                const int m0 = m * kTile + (int)rank * kHalf, n0 = n * kTile + (int)rank * kHalf;
                for (int k = 0; k < p.kb; ++k, ++it) {
                    const uint32_t s = it % kStages, ph = (it / kStages) & 1;
                    if (!wait(empty + 8 * s, ph ^ 1)) { ok = false; break; }
                    const uint32_t bar = map_to_rank(full + 8 * s, 0);
                    if (rank == 0) mbar_expect_tx(full + 8 * s, 2 * kStageBytes);
                    const uint32_t sa = base + s * kStageBytes;
                    load_2d(sa, &maps.x, k * kDepth, m0, bar);
                    load_2d(sa + kStageBytes / 2, &maps.w, k * kDepth, n0, bar);
                }
            }
            // no copy and no arrival may come after the CTA has left: the last fills of the stages are read first
            const uint32_t n = it < (uint32_t)kStages ? it : kStages;
            for (uint32_t j = it - n; j < it && ok; ++j) ok = wait(empty + 8 * (j % kStages), (j / kStages) & 1);
            if (!ok) {   // given up: copies in flight get 10 ms to land
                const uint64_t t0 = globaltimer_ns();
                while (globaltimer_ns() - t0 < 10000000ull) __nanosleep(1000);
            }
        }
    } else if (warp == 1) {
        if (rank == 0 && lane == 0) {
            uint32_t it = 0;
            bool ok = true;
            constexpr uint32_t idesc = idesc_e4m3(kTile, kTile);
            for (int t = pair_id; t < tiles && ok; t += pairs) {
                for (int k = 0; k < p.kb; ++k, ++it) {
                    const uint32_t s = it % kStages, buf = it & 1;
                    if (!wait(acc_empty + 8 * buf, ((it >> 1) & 1) ^ 1) || !wait(full + 8 * s, (it / kStages) & 1)) {
                        ok = false;
                        break;
                    }
                    fence_after_sync();
                    const uint32_t sa = base + s * kStageBytes, sb = sa + kStageBytes / 2;
#pragma unroll
                    for (uint32_t j = 0; j < kDepth / 32; ++j)
                        mma_fp8_pair(tmem + buf * kTile, smem_desc(sa + j * 32, 16, 1024), smem_desc(sb + j * 32, 16, 1024),
                                     idesc, j > 0);
                    commit_pair(empty + 8 * s);
                    commit_pair(acc_full + 8 * buf);
                }
            }
        }
    } else {
        const uint32_t quarter = warp & 3, side = (warp - 2) >> 2;   // the 32 lanes a warp may read; its 128 columns
        const uint32_t buf_s = stores + (warp - 2) * kStore;
        const uint32_t leader_empty = map_to_rank(acc_empty, 0);
        uint32_t it = 0;
        bool ok = true;
        for (int t = pair_id; t < tiles && ok; t += pairs) {
            int m, n;
            pair_tile(p, t, m, n);
            const int row0 = m * kTile + (int)rank * kHalf + (int)quarter * 32;
            const int col0 = n * kTile + (int)side * kHalf;
            const float *xs = p.xs + (int64_t)min(row0 + lane, p.M - 1) * p.kb;
            const float *ws = p.ws + (int64_t)(min(col0, p.N - 1) / kFp8Block) * p.kb;
            Pair acc[64];
#pragma unroll
            for (int i = 0; i < 64; ++i) acc[i] = 0;
            // the scales come two blocks ahead
            float x_now = __ldg(xs), w_now = __ldg(ws), x_next = 0.f, w_next = 0.f;
            if (p.kb > 1) {
                x_next = __ldg(xs + 1);
                w_next = __ldg(ws + 1);
            }
            for (int k = 0; k < p.kb; ++k, ++it) {
                const Pair scale = both(x_now * w_now);
                x_now = x_next;
                w_now = w_next;
                if (k + 2 < p.kb) {
                    x_next = __ldg(xs + k + 2);
                    w_next = __ldg(ws + k + 2);
                }
                const uint32_t buf = it & 1;
                ok = __all_sync(0xffffffffu, wait(acc_full + 8 * buf, (it >> 1) & 1));
                if (!ok) break;
                fence_after_sync();
                const uint32_t src = tmem + buf * kTile + side * kHalf + (quarter << 21);   // lane field: bits 16 and up
#pragma unroll
                for (int ch = 0; ch < 8; ++ch) {
                    uint32_t r[16];
                    tmem_ld16(src + ch * 16, r);
                    wait_ld(r);
                    if (ch == 7) {   // the accumulator is in registers: the next block but one may have it
                        fence_before_sync();
                        __syncwarp();
                        if (lane == 0) arrive_remote_relaxed(leader_empty + 8 * buf);
                    }
#pragma unroll
                    for (int i = 0; i < 8; ++i) acc[8 * ch + i] = fma2(pair_of(r[2 * i], r[2 * i + 1]), scale, acc[8 * ch + i]);
                }
            }
            if (!ok) break;
            // the buffer is written again once the last stores have read it
            if (lane == 0) bulk_wait_read();
            __syncwarp();
#pragma unroll
            for (int j = 0; j < 16; ++j) {   // 8 columns each; 128-byte rows, two boxes
                uint32_t w[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float a, b;
                    split(acc[4 * j + i], a, b);
                    w[i] = pack_bf16(a, b);
                }
                st_shared16(buf_s + (j >> 3) * 4096 + lane * 128 + (((j & 7) ^ (lane & 7)) << 4), w[0], w[1], w[2], w[3]);
            }
            if (p.N % 8 != 0) {   // rows that TMA cannot address: 64 bytes of a row at a time
                __syncwarp();
                const int rows = min(32, p.M - row0);
#pragma unroll 1
                for (int i = lane; i < rows * 128; i += 32) {
                    const int r = i >> 7, c = i & 127;
                    unsigned short v;
                    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v)
                                 : "r"(buf_s + (c >> 6) * 4096 + r * 128 + ((((c & 63) >> 3) ^ (r & 7)) << 4) + (c & 7) * 2));
                    if (col0 + c < p.N) p.out[(int64_t)(row0 + r) * p.N + col0 + c] = __ushort_as_bfloat16(v);
                }
                __syncwarp();
                continue;
            }
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) {
                if (row0 < p.M) {
                    if (col0 < p.N) store_2d(&maps.out, buf_s, col0, row0);
                    if (col0 + 64 < p.N) store_2d(&maps.out, buf_s + 4096, col0 + 64, row0);
                }
                bulk_commit();
            }
        }
        if (lane == 0) bulk_wait_all();
    }
    __syncwarp();
    fence_before_sync();
    __syncthreads();
    cluster_sync();
    fence_after_sync();
    if (warp == 1)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" :: "r"(tmem), "r"(512u) : "memory");
    if (*abort_flag)   // NaN in this CTA's half of each of the pair's tiles
        for (int t = pair_id; t < tiles; t += pairs) {
            int m, n;
            pair_tile(p, t, m, n);
            const int64_t row0 = (int64_t)m * kTile + rank * kHalf;
            for (int i = threadIdx.x; i < kHalf * kTile; i += kPairThreads) {
                const int64_t row = row0 + i / kTile, col = (int64_t)n * kTile + i % kTile;
                if (row < p.M && col < p.N) p.out[row * p.N + col] = __ushort_as_bfloat16(kNaN);
            }
        }
}

// ---------------------------------------------------------------------------
// few tokens
// ---------------------------------------------------------------------------

constexpr int kRows = 128;                  // words of a tile
constexpr int kTable = 4096;                // scales kept at a time
constexpr int kPitch = kRows + 4;           // of the partial sums [token][word]
constexpr int kMostSplits = 8;
constexpr int kMostSmem = 226 * 1024;

template <int TN> constexpr int few_warps() { return TN == 128 ? 8 : 4; }
template <int TN> constexpr int few_threads() { return 64 + 32 * few_warps<TN>(); }
constexpr int few_stage_bytes(int tn) { return (kRows + tn) * kDepth; }
__host__ __device__ constexpr int few_smem(int tn, int stages)
{
    const int data = stages * few_stage_bytes(tn), sums = tn * kPitch * 4;   // the sums take the stages' place
    return 1024 + (data > sums ? data : sums) + kTable * 4 + 16 * stages + 64;
}

__device__ __forceinline__ float4 ld_cluster(uint32_t addr)
{
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
    return v;
}

__device__ __forceinline__ int ld_cluster_int(uint32_t addr)
{
    int v;
    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}

// TN tokens a tile.  The grid: clusters of p.splits CTAs, one a tile, the tiles of the same words next to each other.
template <int TN>
__global__ void __launch_bounds__(few_threads<TN>(), TN == 128 ? 1 : 2) few_kernel(const __grid_constant__ Fp8Maps maps, const __grid_constant__ Fp8Params p)
{
    constexpr int kWarps = few_warps<TN>(), kThreads = few_threads<TN>();
    constexpr int kMine = TN * 4 / kWarps;             // tokens that an epilogue thread sums
    constexpr int kChunk = kMine < 32 ? kMine : 32;
    constexpr uint32_t kCols = TN < 16 ? 32 : 2 * TN;  // of tensor memory
    extern __shared__ unsigned char smem_raw[];
    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    unsigned char *gen = smem_raw + (base - smem_u32(smem_raw));
    const int stage_bytes = few_stage_bytes(TN), stages = p.stages;
    const int data = max(stages * stage_bytes, TN * kPitch * 4);
    float *table = reinterpret_cast<float *>(gen + data);
    float *sums = reinterpret_cast<float *>(gen);
    const uint32_t full = base + data + kTable * 4, empty = full + 8 * stages, acc_full = empty + 8 * stages;
    const uint32_t acc_empty = acc_full + 16, tmem_slot = acc_empty + 16, abort_addr = tmem_slot + 4;
    volatile int *abort_flag = reinterpret_cast<volatile int *>(gen + (abort_addr - base));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int splits = p.splits, rank = (int)(blockIdx.x % (unsigned)splits), tile = (int)(blockIdx.x / (unsigned)splits);
    const int m0 = tile % p.mt * TN, n0 = tile / p.mt * kRows;
    const int k0 = (int)((int64_t)p.kb * rank / splits), k1 = (int)((int64_t)p.kb * (rank + 1) / splits);
    auto wait = [&](uint32_t bar, uint32_t parity) { return wait_here(bar, parity, abort_flag, p); };

    if (threadIdx.x == 32) {
        prefetch_tmap(&maps.x);
        prefetch_tmap(&maps.w);
    }
    if (threadIdx.x == 0) {
        for (int i = 0; i < stages; ++i) {
            mbar_init(full + 8 * i, 1);
            mbar_init(empty + 8 * i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(acc_full + 8 * i, 1);
            mbar_init(acc_empty + 8 * i, kWarps);
        }
        fence_mbar_init();
        *abort_flag = 0;
    }
    if (warp == 1) tmem_alloc(reinterpret_cast<uint32_t *>(gen + (tmem_slot - base)), kCols);
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(gen + (tmem_slot - base));
    start_next();
    wait_previous();
    if (threadIdx.x == 0 && blockIdx.x == 0) *p.err = kDevErrNone;   // a timeout comes a second later at the earliest

    if (warp == 0) {
        if (lane == 0) {
            bool ok = true;
            int it = 0;
            for (int k = (int)blockIdx.x == p.silent ? k1 : k0; k < k1; ++k, ++it) {
                const int s = it % stages;
                if (!wait(empty + 8 * s, ((it / stages) & 1) ^ 1)) { ok = false; break; }
                mbar_expect_tx(full + 8 * s, stage_bytes);
                const uint32_t sa = base + s * stage_bytes;
                tma_load_2d(sa, &maps.w, k * kDepth, n0, full + 8 * s);
                tma_load_2d(sa + kRows * kDepth, &maps.x, k * kDepth, m0, full + 8 * s);
            }
            if (!ok) {   // given up: copies in flight get 10 ms to land
                const uint64_t t0 = globaltimer_ns();
                while (globaltimer_ns() - t0 < 10000000ull) __nanosleep(1000);
            }
        }
    } else if (warp == 1) {
        if (lane == 0) {
            constexpr uint32_t idesc = idesc_e4m3(kRows, TN);
            int it = 0;
            for (int k = k0; k < k1; ++k, ++it) {
                const int s = it % stages;
                const uint32_t buf = it & 1;
                if (!wait(acc_empty + 8 * buf, ((it >> 1) & 1) ^ 1) || !wait(full + 8 * s, (it / stages) & 1)) break;
                fence_after_sync();
                const uint32_t sa = base + s * stage_bytes, sb = sa + kRows * kDepth;
#pragma unroll
                for (uint32_t j = 0; j < kDepth / 32; ++j)
                    mma_fp8(tmem + buf * TN, smem_desc(sa + j * 32, 16, 1024), smem_desc(sb + j * 32, 16, 1024), idesc, j > 0);
                commit(empty + 8 * s);
                commit(acc_full + 8 * buf);
            }
        }
    } else {
        const uint32_t quarter = warp & 3, side = (warp - 2) >> 2;
        const int mine0 = (int)side * kMine, word = (int)quarter * 32 + lane;
        const float *ws = p.ws + (int64_t)(n0 / kFp8Block) * p.kb;
        constexpr int kAhead = kTable / TN;                 // blocks whose scales the table holds
        Pair acc[kMine / 2];
#pragma unroll
        for (int i = 0; i < kMine / 2; ++i) acc[i] = 0;
        bool ok = true;
        int it = 0;
        for (int k = k0; k < k1; ++k, ++it) {
            if (it % kAhead == 0) {   // every warp comes by here, one that has given up too
                const int count = min(kAhead, k1 - k);
                asm volatile("bar.sync 1, %0;" :: "n"(32 * kWarps) : "memory");
                for (int i = threadIdx.x - 64; i < count * TN; i += 32 * kWarps) {
                    const int j = i / count, b = i - j * count;
                    table[b * TN + j] = m0 + j < p.M ? __ldg(p.xs + (int64_t)(m0 + j) * p.kb + k + b) * __ldg(ws + k + b) : 0.f;
                }
                asm volatile("bar.sync 1, %0;" :: "n"(32 * kWarps) : "memory");
            }
            const uint32_t buf = it & 1;
            if (ok) ok = __all_sync(0xffffffffu, wait(acc_full + 8 * buf, (it >> 1) & 1));
            if (!ok) continue;
            fence_after_sync();
            const uint32_t src = tmem + buf * TN + mine0 + (quarter << 21);   // lane field: bits 16 and up
            const ulonglong2 *scale = reinterpret_cast<const ulonglong2 *>(table + it % kAhead * TN + mine0);
#pragma unroll
            for (int ch = 0; ch < kMine / kChunk; ++ch) {
                uint32_t r[kChunk];
                if constexpr (kChunk == 32) tmem_ld32(src + ch * 32, r);
                else tmem_ld16(src + ch * 16, r);
                wait_ld(r);
                if (ch == kMine / kChunk - 1) {
                    fence_before_sync();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(acc_empty + 8 * buf);
                }
#pragma unroll
                for (int i = 0; i < kChunk / 4; ++i) {
                    const ulonglong2 s = scale[ch * (kChunk / 4) + i];
                    Pair *a = acc + ch * (kChunk / 2) + 2 * i;
                    a[0] = fma2(pair_of(r[4 * i], r[4 * i + 1]), s.x, a[0]);
                    a[1] = fma2(pair_of(r[4 * i + 2], r[4 * i + 3]), s.y, a[1]);
                }
            }
        }
        // every product of this CTA is done, so the stages' place is free (or the call has given up: NaN below)
        asm volatile("bar.sync 1, %0;" :: "n"(32 * kWarps) : "memory");
#pragma unroll
        for (int i = 0; i < kMine / 2; ++i) {
            float a, b;
            split(acc[i], a, b);
            sums[(mine0 + 2 * i) * kPitch + word] = a;
            sums[(mine0 + 2 * i + 1) * kPitch + word] = b;
        }
    }
    __syncwarp();
    fence_before_sync();
    __syncthreads();
    if (splits > 1) cluster_sync();
    fence_after_sync();
    if (warp == 1) tmem_dealloc(tmem, kCols);
    bool failed = false;
    for (int r = 0; r < splits; ++r) failed |= ld_cluster_int(map_to_rank(abort_addr, r)) != 0;
    // this CTA's tokens: the partial sums of all, in order
    const int tokens = min(TN, p.M - m0), words = min(kRows, p.N - n0);
    const bool wide = p.N % 8 == 0;
    for (int i = threadIdx.x; i < (tokens + splits - 1 - rank) / splits * 16; i += kThreads) {
        const int j = i / 16 * splits + rank, c = i % 16 * 8;
        if (c >= words) continue;
        float v[8] = {};
        for (int r = 0; r < splits; ++r) {
            const uint32_t at = map_to_rank(base + (uint32_t)(j * kPitch + c) * 4, r);
            const float4 a = ld_cluster(at), b = ld_cluster(at + 16);
            v[0] += a.x; v[1] += a.y; v[2] += a.z; v[3] += a.w;
            v[4] += b.x; v[5] += b.y; v[6] += b.z; v[7] += b.w;
        }
        if (failed)
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = __uint_as_float(0x7fffffffu);
        __nv_bfloat16 *to = p.out + (int64_t)(m0 + j) * p.N + n0 + c;
        if (wide)
            *reinterpret_cast<uint4 *>(to) = make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]),
                                                        pack_bf16(v[6], v[7]));
        else
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (c + e < words) to[e] = __float2bfloat16_rn(v[e]);
    }
    if (splits > 1) cluster_sync();   // nobody leaves while its sums are being read
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

// [rows, K] bytes in 128-B swizzled boxes of box_rows x 128
bool operand_map(CUtensorMap *m, const void *base, int K, int rows, int box_rows)
{
    auto fn = encode_fn();
    if (!fn) return false;
    cuuint64_t dims[2] = {(cuuint64_t)K, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)K};
    cuuint32_t box[2] = {(cuuint32_t)kDepth, (cuuint32_t)box_rows}, es[2] = {1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(base), dims, strides, box, es,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool out_map(CUtensorMap *m, void *base, int N, int M)
{
    auto fn = encode_fn();
    if (!fn) return false;
    cuuint64_t dims[2] = {(cuuint64_t)N, (cuuint64_t)M}, strides[1] = {(cuuint64_t)N * 2};
    cuuint32_t box[2] = {64, 32}, es[2] = {1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, base, dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct Plan {
    int tn;        // few_kernel's tokens a tile, 0 for pair_kernel
    int splits, stages;
};

// The kernel, the tile's tokens and the cut of K that take the least time by a model fitted to measurements (microseconds;
// 512 to 16384 words, K 512 to 6144, 1 to 1024 tokens): a kernel's start and end, more with more tokens a tile and for every
// CTA of a cluster whose sums are joined, and the blocks one after another, once for each round of CTAs.  2048 x 6144 on one
// box: 1 token 5.3 (16 tokens a tile, K in 4; uncut 9.3, pairs 9.5), 64 tokens 8.5 (32, 2; 128 tokens a tile 9.1), 256 tokens
// 10.5 (pairs; 13.5 uncut, 19 to 24 where the CTAs need a second round).
Plan plan(int M, int N, int kb)
{
    Plan best = {0, 1, kStages};
    const int64_t rounds = ((int64_t)ceil_div(M, kTile) * ceil_div(N, kTile) + kPairs - 1) / kPairs;
    float least = 4.5f + rounds * kb * 0.4f;
    for (int tn = 16; tn <= 128; tn *= 2) {
        if (tn < 128 && (M > 4 * tn || (tn > 16 && M <= tn / 2))) continue;
        const int64_t tiles = (int64_t)ceil_div(M, tn) * ceil_div(N, kRows);
        for (int splits = 1; splits <= (tn == 128 ? kMostSplits / 2 : kMostSplits) && splits <= kb; splits *= 2) {
            const int64_t ctas = tiles * splits;
            // two CTAs an SM, but for 128 tokens; clusters of 4 and 8 do not fill every GPC
            const int at_once = (tn == 128 ? 152 : 304) * (splits == 8 ? 27 : splits == 4 ? 30 : 32) / 32;
            const float waves = (float)((ctas + at_once - 1) / at_once);
            const float start = tn == 16 ? 4.f : tn == 32 ? 4.6f : tn == 64 ? 5.4f : 6.2f;
            const float t = waves * (start + ceil_div(kb, splits) * (ctas > 152 ? 0.41f : 0.34f)) + 0.006f * tn * (splits > 1 ? splits : 0);
            if (t >= least) continue;
            least = t;
            const int room = (tn == 128 || (ctas <= 120 && splits <= 4) ? 180 : 88) * 1024;
            const int most = room / few_stage_bytes(tn), need = ceil_div(kb, splits);
            best = {tn, splits, need < most ? need : most};
        }
    }
    return best;
}

template <int TN>
cudaError_t launch_few(const Fp8Maps &maps, const Fp8Params &p, cudaStream_t st)
{
    const int smem = few_smem(TN, p.stages);
    // the same limit whatever this launch takes: another thread's launch may come between the two calls
    const cudaError_t e = cudaFuncSetAttribute(few_kernel<TN>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostSmem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(p.mt * p.nt * p.splits));
    cfg.blockDim = dim3(few_threads<TN>());
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at[2] = {};
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = (unsigned)p.splits;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, few_kernel<TN>, maps, p);
}

}  // namespace

bool fp8_linear_tc_supported(const Fp8LinearArgs &a)
{
    return a.K % 16 == 0 && (((uintptr_t)a.x | (uintptr_t)a.w | (uintptr_t)a.out) & 15) == 0;
}

cudaError_t launch_fp8_linear_tc(const Fp8LinearArgs &a, cudaStream_t st, uint64_t stall_ns)
{
    Fp8Params p = {};
    p.silent = stall_ns ? 0 : -1;
    p.limit_ns = stall_ns ? stall_ns : kWaitLimitNs;
    p.M = a.M; p.N = a.N; p.K = a.K;
    p.kb = ceil_div(a.K, kDepth);
    p.xs = a.xs; p.ws = a.ws;
    p.out = (__nv_bfloat16 *)a.out;
    p.err = (unsigned *)a.workspace;
    const Plan r = plan(a.M, a.N, p.kb);
    p.splits = r.splits;
    p.stages = r.stages;
    p.mt = ceil_div(a.M, r.tn ? r.tn : kTile);
    p.nt = ceil_div(a.N, r.tn ? kRows : kTile);
    Fp8Maps maps;
    memset(&maps, 0, sizeof(maps));
    if (!operand_map(&maps.x, a.x, a.K, a.M, r.tn ? r.tn : kHalf) || !operand_map(&maps.w, a.w, a.K, a.N, kHalf))
        return cudaErrorInvalidValue;
    switch (r.tn) {
    case 16: return launch_few<16>(maps, p, st);
    case 32: return launch_few<32>(maps, p, st);
    case 64: return launch_few<64>(maps, p, st);
    case 128: return launch_few<128>(maps, p, st);
    }
    if (a.N % 8 == 0 && !out_map(&maps.out, a.out, a.N, a.M)) return cudaErrorInvalidValue;
    const cudaError_t e = cudaFuncSetAttribute(pair_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kPairSmem);
    if (e != cudaSuccess) return e;
    const int tiles = p.mt * p.nt, pairs = tiles < kPairs ? tiles : kPairs;
    return launch_early(pair_kernel, 2 * pairs, kPairThreads, kPairSmem, st, maps, p);
}

}  // namespace gdn
