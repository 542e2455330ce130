// gated_scan.cu -- per-channel gated linear recurrence: forward, backward and single-token step.
//
//     h_t = a_t h_{t-1} + c_t x_t,   a = exp(g),   c = 1, or 1 - a with the input gate.
//
// Backward, with e_t = dL/dh_{t-1} (through h_t), a scan from the end of the same form:
//     dH_t = dout_t + e_{t+1},   e_t = a_t dH_t,   e_{len} = dfinal,
//     dx_t = c_t dH_t,           dg_t = a_t dH_t (h_{t-1} [- x_t with the input gate]),   dinit = e_0.
//
// Bound by memory: three tensors forward, five backward (six with the gate), at 3 and 6 operations an element.  What
// keeps the kernel from that bound is the number of instructions an element and the latency of the joins along time,
// hence pairs of channels in one instruction and few, long iterations.  Measured (GB300, bf16, device time): 4 x 2048 x
// 2048, 128 CTAs for 152 SMs, forward 23.5 us (4.3 TB/s), backward 32.5 us (5.2 TB/s); 19 x 2048 x 1024, which fills the
// SMs evenly, forward 39.5 us (6.1 TB/s); 8 packed sequences, 32768 x 2048, forward 92 us (4.4 TB/s; by their lengths 90
// to 100); a step of 256 x 2048 2.1 us.
#include "common.cuh"
#include "kernels.h"
#include "pairs.cuh"

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

__device__ __forceinline__ float exp2_approx(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// exp(g) as 2^(g log2 e) by the hardware's exponential.  In fp32 the rounding of the product g log2 e, |g| / 2 ulp of
// the result, is put back to first order (log2 e as a sum of two floats); for bf16 it stays below the gate's own
// rounding.
template <typename T>
__device__ __forceinline__ Pair decay(Pair g)
{
    const Pair t = mul2(g, pair(1.44269502f, 1.44269502f));
    float t0, t1;
    split(t, t0, t1);
    const float r0 = exp2_approx(t0), r1 = exp2_approx(t1);
    if constexpr (sizeof(T) == 4) {
        const Pair down = mul2(g, pair(-1.44269502f, -1.44269502f));
        const Pair lost = fma2(g, pair(1.92596299e-8f, 1.92596299e-8f), fma2(g, pair(1.44269502f, 1.44269502f), down));
        const Pair r = pair(r0, r1);
        float f0, f1;
        split(fma2(r, mul2(lost, pair(0.693147181f, 0.693147181f)), r), f0, f1);
        // where r is 0 or infinite, or about to be, lost may be NaN
        return pair(fabsf(t0) < 126.f ? f0 : r0, fabsf(t1) < 126.f ? f1 : r1);
    } else {
        return pair(r0, r1);
    }
}

// A lane owns 8 bytes of a row, 4 bf16 or 2 float channels; L lanes (4, 8 or 16) take a row of a CTA's block of
// channels, and the 32 / L groups of a warp take successive runs of R rows.
template <typename T> constexpr int kVec = 8 / sizeof(T);
template <typename T> constexpr int kPairs = kVec<T> / 2;

template <typename T>
__device__ __forceinline__ void unpack(uint2 w, Pair (&v)[kPairs<T>])
{
    if constexpr (sizeof(T) == 4) {
        v[0] = pair(__uint_as_float(w.x), __uint_as_float(w.y));
    } else {
        v[0] = pair(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u));
        v[1] = pair(__uint_as_float(w.y << 16), __uint_as_float(w.y & 0xffff0000u));
    }
}

template <typename T>
__device__ __forceinline__ uint2 pack(const Pair (&v)[kPairs<T>])
{
    float a, b;
    split(v[0], a, b);
    if constexpr (sizeof(T) == 4) {
        return make_uint2(__float_as_uint(a), __float_as_uint(b));
    } else {
        uint2 r;
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r.x) : "f"(b), "f"(a));
        split(v[1], a, b);
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r.y) : "f"(b), "f"(a));
        return r;
    }
}

// One stretch of the recurrence maps a carry c to H + exp(S) c, S the sum of the stretch's g.  exp(S) leaves fp32 from
// |S| = 88 on, although its product with the carry may not; so A is exp(S / 2), and the carry is multiplied by it twice (a
// test for such sums instead cost up to 30 % of the kernel's time).  A is kept finite, so that growth beyond fp32's range
// leaves a carry of 0 at 0; the square of fp32's largest number makes infinity of every other carry that is not subnormal.
template <typename T> struct Map { Pair A[kPairs<T>], H[kPairs<T>]; };

template <typename T>
__device__ __forceinline__ void set_decay(Map<T> &m, const Pair (&sum)[kPairs<T>])
{
#pragma unroll
    for (int v = 0; v < kPairs<T>; ++v) {
        float a, b;
        split(decay<T>(mul2(sum[v], both(0.5f))), a, b);
        m.A[v] = pair(fminf(a, 3.402823466e38f), fminf(b, 3.402823466e38f));
    }
}

// H + A A c
__device__ __forceinline__ Pair through(Pair A, Pair c, Pair H) { return fma2(A, mul2(A, c), H); }

template <typename T>
__device__ __forceinline__ void apply(const Map<T> &m, Pair (&c)[kPairs<T>])
{
#pragma unroll
    for (int v = 0; v < kPairs<T>; ++v) c[v] = through(m.A[v], c[v], m.H[v]);
}

__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__device__ __forceinline__ uint32_t shared_addr(const void *p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }

// The maps of an iteration in shared memory, by turns, so that one barrier an iteration is enough.
template <typename T, int L>
struct Exchange {
    static constexpr int NP = kPairs<T>;
    Map<T> *maps;                   // [2][nwarps][L]: of each warp
    Pair *sums;                     // [2][nwarps][L][pairs]: S of each warp      (cluster only)
    Map<T> *ctas;                   // [2][csize][L]: of each CTA                 (cluster only)
    int nwarps, csize, rank;
    static __host__ __device__ int bytes(int nwarps, int csize)
    {
        return 2 * L * (nwarps * (int)sizeof(Map<T>) + (csize > 1 ? nwarps * NP * 8 + csize * (int)sizeof(Map<T>) : 0));
    }
    __device__ __forceinline__ Exchange(unsigned char *p, int nw, int cs, int rk)
        : maps((Map<T> *)p), sums((Pair *)(maps + 2 * nw * L)), ctas((Map<T> *)(sums + 2 * nw * L * NP)),
          nwarps(nw), csize(cs), rank(rk) {}

    // The work of a cluster's extra warp: joins its CTA's maps and hands the result to the other CTAs.  It stores
    // nothing to global memory: the release that makes the maps visible waits for all earlier stores of its thread,
    // and with the rows' own stores among them that wait took a quarter of the kernel.
    __device__ __forceinline__ void hand_over(int turn)
    {
        const int lane = threadIdx.x & (L - 1);
        __syncthreads();
        Map<T> all;
        Pair s[NP];
#pragma unroll
        for (int v = 0; v < NP; ++v) s[v] = all.H[v] = 0;
        for (int w = 0; w < nwarps; ++w) {
            apply(maps[(turn * nwarps + w) * L + lane], all.H);
#pragma unroll
            for (int v = 0; v < NP; ++v) s[v] = add2(s[v], sums[((turn * nwarps + w) * L + lane) * NP + v]);
        }
        set_decay<T>(all, s);
        // the groups of the warp share the CTAs out
        const uint32_t mine = shared_addr(&ctas[(turn * csize + rank) * L + lane]);
        for (int r = (threadIdx.x & 31) / L; r < csize; r += 32 / L) {
            uint32_t to;
            asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(to) : "r"(mine), "r"(r));
#pragma unroll
            for (int v = 0; v < NP; ++v) {
                asm volatile("st.shared::cluster.b64 [%0], %1;" :: "r"(to + 8 * v), "l"(all.A[v]) : "memory");
                asm volatile("st.shared::cluster.b64 [%0], %1;" :: "r"(to + 8 * (NP + v)), "l"(all.H[v]) : "memory");
            }
        }
        __syncwarp();
        cluster_sync();
    }

    // On entry a group holds the sum S and the map's H of its rows, and every thread the carry into the iteration's
    // first row; returns the carry into the group's rows and moves `carry` behind the iteration's last row.  The order
    // is fixed: groups, warps, CTAs.
    template <bool CLUSTER>
    __device__ __forceinline__ void join(int turn, Pair (&s)[NP], Pair (&h)[NP], Pair (&carry)[NP], Pair (&in)[NP])
    {
        const int lane = threadIdx.x & (L - 1), group = (threadIdx.x & 31) / L, warp = threadIdx.x >> 5;
        Map<T> m;
        // scan over the warp's groups: each takes in the ones before it, 1, 2, 4 at a time
#pragma unroll
        for (int o = 1; o < 32 / L; o *= 2) {
            set_decay<T>(m, s);
#pragma unroll
            for (int v = 0; v < NP; ++v) {
                const Pair so = __shfl_up_sync(0xffffffffu, s[v], o * L), ho = __shfl_up_sync(0xffffffffu, h[v], o * L);
                if (group >= o) {
                    h[v] = through(m.A[v], ho, h[v]);
                    s[v] = add2(s[v], so);
                }
            }
        }
        if (group == 32 / L - 1) {
            set_decay<T>(m, s);
#pragma unroll
            for (int v = 0; v < NP; ++v) m.H[v] = h[v];
            maps[(turn * nwarps + warp) * L + lane] = m;
            if (CLUSTER)
#pragma unroll
                for (int v = 0; v < NP; ++v) sums[((turn * nwarps + warp) * L + lane) * NP + v] = s[v];
        }
        // the map of the groups before this one
        Map<T> before;
#pragma unroll
        for (int v = 0; v < NP; ++v) {
            s[v] = __shfl_up_sync(0xffffffffu, s[v], L & 31);
            before.H[v] = __shfl_up_sync(0xffffffffu, h[v], L & 31);
        }
        set_decay<T>(before, s);
        __syncthreads();
        const Map<T> *all = maps + turn * nwarps * L + lane;
        if (CLUSTER) {
            asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
            asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
            for (int r = 0; r < csize; ++r) {
#pragma unroll
                for (int v = 0; v < NP; ++v) in[v] = r == rank ? carry[v] : in[v];
                apply(ctas[(turn * csize + r) * L + lane], carry);
            }
#pragma unroll 4
            for (int w = 0; w < warp; ++w) apply(all[w * L], in);
        } else {
#pragma unroll 4
            for (int w = 0; w < warp; ++w) apply(all[w * L], carry);
#pragma unroll
            for (int v = 0; v < NP; ++v) in[v] = carry[v];
#pragma unroll 4
            for (int w = warp; w < nwarps; ++w) apply(all[w * L], carry);
        }
        if (group > 0) apply(before, in);
    }
};

// How rows get into shared memory, by their alignment (device time of the backward pass, bf16, N x T x D).
//   kWhole    every row starts on a 16-byte boundary: copies of 16 bytes.
//   kWords    bf16, every row on a 4-byte boundary: copies of 4 bytes.
//   kShifted  rows anywhere in tensors that start on 16-byte boundaries: the 16-byte chunks that hold a row are copied,
//             and it is read where it lies in them.  4 x 2048 x 2049: 57 us, element by element 249; fp32 4 x 2048 x
//             1001: 42 us, by words 64.  For rows that words fit, the three reads of each lane cost bf16 more than
//             they save: 8 x 28544 x 26 124 us, by words 62; 4 x 2048 x 2050 57 and 68, forward 39 and 34.
//   kElements anything else: element by element through registers.
enum { kWhole = 16, kWords = 4, kShifted = 1, kElements = 2 };

// A warp's slot: its rows, R of a group together, and a gap after each group of short rows, so that the groups, which
// read one row each, find theirs in different banks (without it the backward pass of 1 x 4999 x 1001 waited on shared
// memory more than on anything else).
template <int L, int R, int CW>
struct Slot {
    static constexpr int kPitch = 8 * L + (CW == kShifted ? 16 : 0);
    static constexpr int kPad = L < 16 ? ((8 * L - R * kPitch) % 128 + 128) % 128 : 0;
    static constexpr int kGroup = R * kPitch + kPad;
    static constexpr int kBytes = (kGroup * (32 / L) + 127) / 128 * 128;
    static __device__ __forceinline__ uint32_t at(int row) { return row * kPitch + row / R * kPad; }
    // row r0 + down * i, where down is a power of two and r0 < down
    template <int DOWN>
    static __device__ __forceinline__ uint32_t at(int r0, int i)
    {
        const int group = DOWN >= R ? r0 / R + i * (DOWN / R) : i * DOWN / R;
        return (r0 + DOWN * i) * kPitch + group * kPad;
    }
};

// A warp's 32 / L groups of R rows into its slot; row i at src + i * step elements, rows from `rows` on as zeros and
// channels behind D as anything; `end` is the tensor's.
template <typename T, int L, int R, int CW, bool WHOLE>
__device__ __forceinline__ void fetch_some(uint32_t slot, const T *src, const T *end, int step, int rows, int channels)
{
    using S = Slot<L, R, CW>;
    constexpr int ROWS = R * 32 / L;
    const int lane = threadIdx.x & 31;
    if constexpr (CW == kWhole) {
        constexpr int across = L / 2, down = 32 / across;   // copies a row; rows a step
        const int col = (lane % across) * (16 / (int)sizeof(T)), r0 = lane / across;
        const T *p = src + ((int64_t)step * r0 + col);
        const bool live = col < channels;
#pragma unroll
        for (int i = 0; i < ROWS / down; ++i) {
            const bool in = WHOLE || (live && r0 + down * i < rows);
            const T *from = p + (int64_t)step * (down * i);   // read if `in`
            asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;"
                         :: "r"(slot + (lane % across) * 16 + S::template at<down>(r0, i)), "l"(from), "r"(in ? 16 : 0)
                         : "memory");
        }
    } else if constexpr (CW == kWords) {
        constexpr int across = L * 2 < 32 ? L * 2 : 32, down = 32 / across, per = 4 / (int)sizeof(T);
        const int col = (lane % across) * per, r0 = lane / across;
        const T *p = src + ((int64_t)step * r0 + col);
        const bool live = col < channels;
#pragma unroll
        for (int i = 0; i < ROWS / down; ++i) {
            const bool in = WHOLE || (live && r0 + down * i < rows);
            const T *from = p + (int64_t)step * (down * i);
            asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;"
                         :: "r"(slot + (lane % across) * 4 + S::template at<down>(r0, i)), "l"(from), "r"(in ? 4 : 0)
                         : "memory");
        }
    } else if constexpr (CW == kShifted) {
        constexpr int across = L / 2 + 1, items = ROWS * across;
#pragma unroll
        for (int i = 0; i < (items + 31) / 32; ++i) {
            const int k = lane + 32 * i, r = k / across, chunk = k - r * across;
            const uintptr_t row = reinterpret_cast<uintptr_t>(src + (int64_t)step * r);
            const uintptr_t from = (row & ~(uintptr_t)15) + 16 * chunk;
            // up to the row's last byte, and no further than the tensor's
            int bytes = 0;
            if (r < rows && from < row + channels * sizeof(T))
                bytes = (int)min((uintptr_t)16, reinterpret_cast<uintptr_t>(end) - from);
            if (items % 32 == 0 || k < items)
                asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;"
                             :: "r"(slot + S::at(r) + 16 * chunk), "l"(from), "r"(bytes) : "memory");
        }
    } else {
        constexpr int across = L * 2 < 32 ? L * 2 : 32, down = 32 / across, per = 4 / (int)sizeof(T);
        const int col = (lane % across) * per, r0 = lane / across;
        uint32_t w[ROWS / down];
#pragma unroll
        for (int i = 0; i < ROWS / down; ++i) {
            const T *p = src + ((int64_t)step * (r0 + down * i) + col);
            const bool in = r0 + down * i < rows;
            w[i] = 0;
            if constexpr (sizeof(T) == 4) {
                if (in && col < channels) w[i] = __ldg(reinterpret_cast<const uint32_t *>(p));
            } else {
                if (in && col < channels) w[i] = __ldg(reinterpret_cast<const unsigned short *>(p));
                if (in && col + 1 < channels) w[i] |= (uint32_t)__ldg(reinterpret_cast<const unsigned short *>(p) + 1) << 16;
            }
        }
#pragma unroll
        for (int i = 0; i < ROWS / down; ++i)
            asm volatile("st.shared.b32 [%0], %1;"
                         :: "r"(slot + (lane % across) * 4 + S::template at<down>(r0, i)), "r"(w[i]) : "memory");
    }
}

// Nearly all of them are whole: those go without the tests, a third of the instructions of the 4-byte copies.
template <typename T, int L, int R, int CW>
__device__ __forceinline__ void fetch(uint32_t slot, const T *src, const T *end, int step, int rows, int channels)
{
    if ((CW == kWhole || CW == kWords) && rows == R * 32 / L && channels == L * kVec<T>)
        fetch_some<T, L, R, CW, true>(slot, src, end, step, rows, channels);
    else
        fetch_some<T, L, R, CW, false>(slot, src, end, step, rows, channels);
}

// The lane's channels of one row, out of a slot.  shift: where the row starts in its first chunk (kShifted).
template <typename T, int CW>
__device__ __forceinline__ uint2 words(uint32_t at, uint32_t shift)
{
    uint2 w;
    if constexpr (CW != kShifted) {
        asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(w.x), "=r"(w.y) : "r"(at));
    } else if constexpr (sizeof(T) == 4) {
        asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w.x) : "r"(at + shift));
        asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w.y) : "r"(at + shift + 4));
    } else {
        const uint32_t from = at + (shift & ~3u);
        uint32_t a, b, c = 0;
        asm volatile("ld.shared.b32 %0, [%1];" : "=r"(a) : "r"(from));
        asm volatile("ld.shared.b32 %0, [%1];" : "=r"(b) : "r"(from + 4));
        asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %2, 0;\n\t@p ld.shared.b32 %0, [%1];\n\t}"
                     : "+r"(c) : "r"(from + 8), "r"(shift & 2));
        w.x = __funnelshift_r(a, b, (shift & 2) * 8);
        w.y = __funnelshift_r(b, c, (shift & 2) * 8);
    }
    return w;
}

// The lane's channels of one row; `mine` = how many of them lie before D.  WHOLE: all of the group's.
template <typename T, int L, int CW, bool WHOLE>
__device__ __forceinline__ void put(T *dst, const Pair (&v)[kPairs<T>], int mine)
{
    const uint2 w = pack<T>(v);
    if constexpr (CW == kWhole) {
        if (WHOLE || mine > 0) *reinterpret_cast<uint2 *>(dst) = w;
    } else if constexpr (sizeof(T) == 4 || CW == kWords) {
        constexpr int per = 4 / sizeof(T);
        if (WHOLE || mine > 0) *reinterpret_cast<uint32_t *>(dst) = w.x;
        if (WHOLE || mine > per) *reinterpret_cast<uint32_t *>(dst + per) = w.y;
    } else if constexpr (WHOLE) {
        // a row at an odd element: its words are made of neighbours, the last one with the next lane's first
        const int lane = threadIdx.x & (L - 1);
        const uint32_t next = __shfl_down_sync(0xffffffffu, w.x, 1);
        if ((reinterpret_cast<uintptr_t>(dst) & 2) == 0) {
            *reinterpret_cast<uint32_t *>(dst) = w.x;
            *reinterpret_cast<uint32_t *>(dst + 2) = w.y;
        } else {
            unsigned short *p = reinterpret_cast<unsigned short *>(dst);
            if (lane == 0) p[0] = (unsigned short)w.x;
            *reinterpret_cast<uint32_t *>(dst + 1) = __funnelshift_r(w.x, w.y, 16);
            if (lane < L - 1) *reinterpret_cast<uint32_t *>(dst + 3) = __funnelshift_r(w.y, next, 16);
            else p[3] = (unsigned short)(w.y >> 16);
        }
    } else {
        unsigned short *p = reinterpret_cast<unsigned short *>(dst);
        if (mine > 0) p[0] = (unsigned short)w.x;
        if (mine > 1) p[1] = (unsigned short)(w.x >> 16);
        if (mine > 2) p[2] = (unsigned short)w.y;
        if (mine > 3) p[3] = (unsigned short)(w.y >> 16);
    }
}

__device__ __forceinline__ void commit_copies() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void wait_copies() { asm volatile("cp.async.wait_group %0;" :: "n"(N) : "memory"); }

// The k-th longest of up to 32 packed sequences (the first of equals): the long ones start first.
__device__ __forceinline__ int by_length(const GatedScanArgs &a, int k)
{
    const int lane = threadIdx.x & 31;
    const int len = lane < a.N ? __ldg(a.cu + lane + 1) - __ldg(a.cu + lane) : -1;
    int longer = 0;
    for (int i = 0; i < a.N; ++i) {
        const int other = __shfl_sync(0xffffffffu, len, i);
        longer += other > len || (other == len && i < lane);
    }
    return __ffs(__ballot_sync(0xffffffffu, lane < a.N && longer == k)) - 1;
}

struct Yes { __device__ constexpr bool operator()() const { return true; } };
struct No { __device__ constexpr bool operator()() const { return false; } };

// What a CTA works on: one sequence (with the cluster's other CTAs, along time) and one block of L kVec channels.
template <typename T, int L>
struct Work {
    int n, ch0, channels, rank, len, mine;
    int64_t tok0, total;   // the first token; elements of a tensor
    __device__ __forceinline__ Work(const GatedScanArgs &a, int nblocks, int csize)
    {
        rank = blockIdx.x % csize;
        const int unit = blockIdx.x / csize;
        n = unit / nblocks;
        if (a.cu && a.N <= 32) n = by_length(a, n);
        ch0 = (unit % nblocks) * (L * kVec<T>);
        channels = min(a.D - ch0, (L * kVec<T>));
        mine = channels - (threadIdx.x & (L - 1)) * kVec<T>;
        span(a, n, tok0, len);
        total = (int64_t)(a.cu ? 1 : a.N) * a.T * a.D;
    }
    // whether all the warp's groups have all their rows and channels
    __device__ __forceinline__ bool whole(int rows, int most) const
    {
        return channels == L * kVec<T> && __all_sync(0xffffffffu, rows == most);
    }
    __device__ __forceinline__ void get(const float *s, const GatedScanArgs &a, Pair (&p)[kPairs<T>]) const
    {
        const float *at = s + (int64_t)n * a.D + ch0 + (threadIdx.x & (L - 1)) * kVec<T>;
#pragma unroll
        for (int v = 0; v < kPairs<T>; ++v)
            p[v] = pair(s && 2 * v < mine ? at[2 * v] : 0.f, s && 2 * v + 1 < mine ? at[2 * v + 1] : 0.f);
    }
    __device__ __forceinline__ void set(float *s, const GatedScanArgs &a, const Pair (&p)[kPairs<T>]) const
    {
        float *at = s + (int64_t)n * a.D + ch0 + (threadIdx.x & (L - 1)) * kVec<T>;
#pragma unroll
        for (int v = 0; v < kPairs<T>; ++v) {
            float x, y;
            split(p[v], x, y);
            if (s && 2 * v < mine) at[2 * v] = x;
            if (s && 2 * v + 1 < mine) at[2 * v + 1] = y;
        }
    }
};

__device__ __forceinline__ int rows_left(int64_t from, int len, int most)
{
    return (int)max((int64_t)0, min((int64_t)most, len - from));
}

// 1 - exp(g), given a = exp(g): the series of exp(g) - 1 where |g| <= 1/2 and the difference would lose bits (the next
// term is under 2^-26 of the sum), else the difference.
__device__ __forceinline__ Pair gate_of(Pair g, Pair a)
{
    Pair s = both(1.f / 40320.f);
    s = fma2(s, g, both(1.f / 5040.f));
    s = fma2(s, g, both(1.f / 720.f));
    s = fma2(s, g, both(1.f / 120.f));
    s = fma2(s, g, both(1.f / 24.f));
    s = fma2(s, g, both(1.f / 6.f));
    s = fma2(s, g, both(0.5f));
    s = fma2(s, g, both(1.f));
    float g0, g1, a0, a1, s0, s1;
    split(g, g0, g1);
    split(a, a0, a1);
    split(mul2(s, g), s0, s1);
    return pair(fabsf(g0) <= 0.5f ? -s0 : 1.f - a0, fabsf(g1) <= 0.5f ? -s1 : 1.f - a1);
}

// CTAs that registers are limited for.  Copies by words hold so many addresses that 128 registers spill over them:
// backward 1 x 25951 x 1546 364 us with two CTAs' registers, 215 with one's, 4 x 2048 x 2050 68 and 52; forward 141 and
// 126 with 4 lanes a row, but 32 and 35 (16 x 1000 x 1002) with 16.
constexpr int ctas_an_sm(bool backward, bool gate, int cw, int L, int R, bool cluster)
{
    return cluster || (backward && gate && R == 8) || (cw == kWords && (backward || L == 4)) ? 1 : 2;
}

// An iteration takes csize * nwarps * R * 32 / L rows.  Rows pass through a ring of each warp's own slots by asynchronous
// copies, so only the joins need barriers.  A group scans its R rows from 0 (S and H), the joined carry comes in,
// and the rows are run again from it out of registers: memory is read once and written once.
template <typename T, bool GATE, int CW, int L, int R, int STAGES, int WARPS, bool CLUSTER>
__global__ void __launch_bounds__(32 * WARPS + (CLUSTER ? 32 : 0), ctas_an_sm(false, GATE, CW, L, R, CLUSTER))
scan_fwd_kernel(const GatedScanArgs a, int nblocks, int csize)
{
    constexpr int NP = kPairs<T>, ROWS = R * 32 / L, SLOT = Slot<L, R, CW>::kBytes, PITCH = Slot<L, R, CW>::kPitch;
    extern __shared__ __align__(128) unsigned char smem[];
    const int warp = threadIdx.x >> 5, nwarps = (blockDim.x >> 5) - (CLUSTER ? 1 : 0);
    const Work<T, L> w(a, nblocks, csize);
    Exchange<T, L> ex(smem + nwarps * STAGES * 2 * SLOT, nwarps, csize, w.rank);
    const int64_t per = (int64_t)csize * nwarps * ROWS;
    int turn = 0, stage = 0;
    if (CLUSTER) {
        cluster_sync();   // the others' shared memory may be written once they run
        if (warp == nwarps) {
            for (int64_t first = 0; first < w.len; first += per, turn ^= 1) ex.hand_over(turn);
            return;
        }
    }

    const uint32_t slots = shared_addr(smem) + warp * STAGES * 2 * SLOT;
    const int group = (threadIdx.x & 31) / L;
    const uint32_t own = group * Slot<L, R, CW>::kGroup + (threadIdx.x & (L - 1)) * 8;
    const int64_t base = w.tok0 * a.D + w.ch0, total = w.total;
    Pair carry[NP];
    w.get(a.init_state, a, carry);
    int64_t t0 = (int64_t)(w.rank * nwarps + warp) * ROWS;   // the warp's first row of the iteration
    auto load = [&](int64_t t, int st) {
        const int rows = rows_left(t, w.len, ROWS);
        const int64_t at = base + (rows > 0 ? t * a.D : 0);
        fetch<T, L, R, CW>(slots + st * 2 * SLOT, (const T *)a.g + at, (const T *)a.g + total, a.D, rows, w.channels);
        fetch<T, L, R, CW>(slots + (st * 2 + 1) * SLOT, (const T *)a.x + at, (const T *)a.x + total, a.D, rows, w.channels);
    };
#pragma unroll
    for (int s = 0; s < STAGES; ++s) {
        load(t0 + s * per, s);
        commit_copies();
    }
    for (int64_t first = 0; first < w.len; first += per, t0 += per, turn ^= 1) {
        wait_copies<STAGES - 1>();
        __syncwarp();
        const uint32_t sg = slots + stage * 2 * SLOT + own, sx = sg + SLOT;
        // where the group's rows start in their chunks: byte offsets, of which 4 bits matter
        const uint32_t off = (uint32_t)(base + (t0 + group * R) * a.D) * (uint32_t)sizeof(T), inc = (uint32_t)a.D * sizeof(T);
        Pair al[R][NP], u[R][NP], sum[NP], h[NP], in[NP];
#pragma unroll
        for (int v = 0; v < NP; ++v) sum[v] = h[v] = 0;
#pragma unroll
        for (int i = 0; i < R; ++i) {
            unpack<T>(words<T, CW>(sg + i * PITCH, (off + i * inc) & 15), al[i]);   // rows behind the end: g = x = 0, the identity
            unpack<T>(words<T, CW>(sx + i * PITCH, (off + i * inc) & 15), u[i]);
#pragma unroll
            for (int v = 0; v < NP; ++v) {
                sum[v] = add2(sum[v], al[i][v]);
                const Pair g = al[i][v];
                al[i][v] = decay<T>(g);
                if (GATE) u[i][v] = mul2(u[i][v], gate_of(g, al[i][v]));
                h[v] = fma2(al[i][v], h[v], u[i][v]);
            }
        }
        __syncwarp();
        load(t0 + STAGES * per, stage);
        commit_copies();
        stage = stage + 1 == STAGES ? 0 : stage + 1;
        ex.template join<CLUSTER>(turn, sum, h, carry, in);
        const int rows = rows_left(t0 + group * R, w.len, R);
        T *out = (T *)a.out + (base + (t0 + group * R) * a.D + (threadIdx.x & (L - 1)) * kVec<T>);
        auto emit = [&](auto whole) {
#pragma unroll
            for (int i = 0; i < R; ++i) {
#pragma unroll
                for (int v = 0; v < NP; ++v) in[v] = fma2(al[i][v], in[v], u[i][v]);
                if (whole() || i < rows) put<T, L, CW, whole()>(out + (int64_t)a.D * i, in, w.mine);
            }
        };
        if (w.whole(rows, R)) emit(Yes());
        else emit(No());
    }
    wait_copies<0>();
    if (w.rank == 0 && warp == 0 && group == 0) w.set(a.final_state, a, carry);
}

// The same from the end: row i of a warp's slot is token len - 1 - (r0 + i), its h the one before.
template <typename T, bool GATE, int CW, int L, int R, int STAGES, int WARPS, bool CLUSTER>
__global__ void __launch_bounds__(32 * WARPS + (CLUSTER ? 32 : 0), ctas_an_sm(true, GATE, CW, L, R, CLUSTER))
scan_bwd_kernel(const GatedScanArgs a, int nblocks, int csize)
{
    constexpr int NP = kPairs<T>, NT = GATE ? 4 : 3, ROWS = R * 32 / L, SLOT = Slot<L, R, CW>::kBytes, PITCH = Slot<L, R, CW>::kPitch;
    extern __shared__ __align__(128) unsigned char smem[];
    const int warp = threadIdx.x >> 5, nwarps = (blockDim.x >> 5) - (CLUSTER ? 1 : 0);
    const Work<T, L> w(a, nblocks, csize);
    Exchange<T, L> ex(smem + nwarps * STAGES * NT * SLOT, nwarps, csize, w.rank);
    const int64_t per = (int64_t)csize * nwarps * ROWS;
    int turn = 0, stage = 0;
    if (CLUSTER) {
        cluster_sync();
        if (warp == nwarps) {
            for (int64_t first = 0; first < w.len; first += per, turn ^= 1) ex.hand_over(turn);
            return;
        }
    }

    const uint32_t slots = shared_addr(smem) + warp * STAGES * NT * SLOT;
    const int group = (threadIdx.x & 31) / L;
    const uint32_t own = group * Slot<L, R, CW>::kGroup + (threadIdx.x & (L - 1)) * 8;
    const int64_t last = (w.tok0 + w.len - 1) * a.D + w.ch0, total = w.total;
    Pair carry[NP];
    w.get(a.dfinal, a, carry);
    int64_t r0 = (int64_t)(w.rank * nwarps + warp) * ROWS;
    auto load = [&](int64_t r, int st) {
        const int rows = rows_left(r, w.len, ROWS), before = rows_left(r, w.len - 1, ROWS);   // the first token has none
        const int64_t at = rows > 0 ? last - r * a.D : 0;
        const uint32_t s = slots + st * NT * SLOT;
        fetch<T, L, R, CW>(s, (const T *)a.g + at, (const T *)a.g + total, -a.D, rows, w.channels);
        fetch<T, L, R, CW>(s + SLOT, (const T *)a.dout + at, (const T *)a.dout + total, -a.D, rows, w.channels);
        fetch<T, L, R, CW>(s + 2 * SLOT, (const T *)a.h + (before > 0 ? at - a.D : 0), (const T *)a.h + total, -a.D, before,
                           w.channels);
        if (GATE) fetch<T, L, R, CW>(s + 3 * SLOT, (const T *)a.x + at, (const T *)a.x + total, -a.D, rows, w.channels);
    };
#pragma unroll
    for (int s = 0; s < STAGES; ++s) {
        load(r0 + s * per, s);
        commit_copies();
    }
    for (int64_t first = 0; first < w.len; first += per, r0 += per, turn ^= 1) {
        wait_copies<STAGES - 1>();
        __syncwarp();
        const uint32_t sg = slots + stage * NT * SLOT + own, sd = sg + SLOT, shh = sd + SLOT, sx = shh + SLOT;
        const uint32_t off = (uint32_t)(last - (r0 + group * R) * a.D) * (uint32_t)sizeof(T), inc = (uint32_t)a.D * sizeof(T);
        Pair al[R][NP], d[R][NP], sum[NP], h[NP], e[NP];
#pragma unroll
        for (int v = 0; v < NP; ++v) sum[v] = h[v] = 0;
#pragma unroll
        for (int i = 0; i < R; ++i) {
            unpack<T>(words<T, CW>(sg + i * PITCH, (off - i * inc) & 15), al[i]);
            unpack<T>(words<T, CW>(sd + i * PITCH, (off - i * inc) & 15), d[i]);
#pragma unroll
            for (int v = 0; v < NP; ++v) {
                sum[v] = add2(sum[v], al[i][v]);
                al[i][v] = decay<T>(al[i][v]);
                h[v] = mul2(al[i][v], add2(h[v], d[i][v]));
            }
        }
        ex.template join<CLUSTER>(turn, sum, h, carry, e);
        const int64_t rh = r0 + group * R;
        const int rows = rows_left(rh, w.len, R);
        const int64_t start = w.len - 1 - rh;   // the row of the sequence's first token
        const int64_t at = last - rh * a.D + (threadIdx.x & (L - 1)) * kVec<T>;
        auto emit = [&](auto whole) {
#pragma unroll
            for (int i = 0; i < R; ++i) {
                Pair prev[NP], x[NP], g[NP], vx[NP], vg[NP];
                unpack<T>(words<T, CW>(shh + i * PITCH, (off - (i + 1) * inc) & 15), prev);
                if (i == start) w.get(a.init_state, a, prev);
                if (GATE) {
                    unpack<T>(words<T, CW>(sx + i * PITCH, (off - i * inc) & 15), x);
                    unpack<T>(words<T, CW>(sg + i * PITCH, (off - i * inc) & 15), g);
                }
#pragma unroll
                for (int v = 0; v < NP; ++v) {
                    const Pair dh = add2(d[i][v], e[v]);
                    e[v] = mul2(al[i][v], dh);
                    vx[v] = GATE ? mul2(gate_of(g[v], al[i][v]), dh) : dh;
                    vg[v] = mul2(e[v], GATE ? fma2(x[v], pair(-1.f, -1.f), prev[v]) : prev[v]);
                }
                if (whole() || i < rows) {
                    put<T, L, CW, whole()>((T *)a.dx + at - (int64_t)a.D * i, vx, w.mine);
                    put<T, L, CW, whole()>((T *)a.dg + at - (int64_t)a.D * i, vg, w.mine);
                }
            }
        };
        if (w.whole(rows, R)) emit(Yes());
        else emit(No());
        __syncwarp();
        load(r0 + STAGES * per, stage);
        commit_copies();
        stage = stage + 1 == STAGES ? 0 : stage + 1;
    }
    wait_copies<0>();
    if (w.rank == 0 && warp == 0 && group == 0) w.set(a.dinit, a, carry);
}

// Eight elements a thread where the arrays allow 16-byte accesses of the element type, else one.
template <typename T, bool GATE, int E>
__global__ void __launch_bounds__(256) scan_step_kernel(float *state, const T *x, const T *g, T *out, int64_t n)
{
    const int64_t stride = (int64_t)gridDim.x * 256 * E;
    for (int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * E; i < n; i += stride) {
        T xv[E], gv[E], ov[E];
        float h[E];
        if constexpr (E == 8) {
            constexpr int Q = E * sizeof(T) / 16;
#pragma unroll
            for (int q = 0; q < Q; ++q) {
                reinterpret_cast<uint4 *>(xv)[q] = __ldcs(reinterpret_cast<const uint4 *>(x + i) + q);
                reinterpret_cast<uint4 *>(gv)[q] = __ldcs(reinterpret_cast<const uint4 *>(g + i) + q);
            }
#pragma unroll
            for (int q = 0; q < 2; ++q)
                reinterpret_cast<float4 *>(h)[q] = *(reinterpret_cast<const float4 *>(state + i) + q);
        } else {
            xv[0] = x[i];
            gv[0] = g[i];
            h[0] = state[i];
        }
#pragma unroll
        for (int j = 0; j < E; ++j) {
            const float gg = to_f32(gv[j]), xx = to_f32(xv[j]);
            h[j] = fmaf(expf(gg), h[j], GATE ? -expm1f(gg) * xx : xx);
            ov[j] = from_f32<T>(h[j]);
        }
        if constexpr (E == 8) {
#pragma unroll
            for (int q = 0; q < 2; ++q)
                *(reinterpret_cast<float4 *>(state + i) + q) = reinterpret_cast<float4 *>(h)[q];
#pragma unroll
            for (int q = 0; q < (int)(E * sizeof(T) / 16); ++q)
                *(reinterpret_cast<uint4 *>(out + i) + q) = reinterpret_cast<uint4 *>(ov)[q];
        } else {
            state[i] = h[0];
            out[i] = ov[0];
        }
    }
}

// How the work is cut: lanes a row, warps a CTA, CTAs a cluster.
//
// An iteration of a CTA takes some 2 us however few rows that is, so what is needed is enough CTAs with many rows each.
// Rows of 128 bytes (16 lanes) come first; where they make fewer than 80 CTAs, narrower ones, whose groups in the warp
// go along time instead, make more CTAs of more rows (device time of the forward pass, bf16, N x T x D, with 16, 8 and
// 4 lanes a row: 64 x 2048 x 512 73, 76, 94 us; 11 x 3292 x 256 36, 21, 21 us; 2 x 4096 x 1024 44, 24, 15 us).  Packed
// sequences of unequal lengths are held up by the longest and take more CTAs (forward, 32768 x 2048 in 8 sequences 146, 99,
// 92 us, in 16 85, 77, 99, in 30 80, 88, 117; 32768 x 1024 in 8 133, 83, 61; backward in 8 198, 141, 145, in 16 127, 110,
// 147).  16 warps a CTA measured slower throughout (2 x 4096 x 1024: 17).
//
// A cluster's join adds 2 to 3 us an iteration (4 x 2048 x 2048 in clusters of two: 75 us instead of 24), so clusters
// serve only where 32-byte rows still leave most SMs idle over a long time, and no more of them than the GPU holds at
// once: a GPC's 16 to 20 SMs fit four clusters of four but two of eight (1 x 32768 x 64, 4 CTAs of rows: 97 us alone,
// 38 in clusters of 4, 25 of 8, 18 of 16; 1 x 16384 x 256, 16 CTAs: 50 alone, 23 of 4, 31 of 8; 1 x 8192 x 512, 32
// CTAs: 26 alone, 23 of 2, 15 of 4, 32 of 8).
struct Cut { int lanes, warps, csize; };

// cluster_warps: as many as shared memory holds, beside the one that hands over
Cut cut(const GatedScanArgs &a, int vec, int R, int cluster_warps)
{
    Cut c = {16, 8, 1};
    const int64_t longest = a.cu ? (3 * (int64_t)a.T / a.N + 1 < a.T ? 3 * (int64_t)a.T / a.N + 1 : a.T) : a.T;
    auto units = [&] { return (int64_t)a.N * ceil_div(a.D, c.lanes * vec); };
    auto rows = [&] { return (int64_t)c.csize * c.warps * R * 32 / c.lanes; };
    while (c.lanes > 4 && units() < (a.cu ? 912 : 80) && rows() < longest) c.lanes /= 2;
    if (c.lanes > 4 || longest <= 4 * rows()) return c;
    const int most[] = {50, 34, 14, 7};   // clusters of 2, 4, 8, 16
    c.warps = cluster_warps;
    for (int i = 0; i < 4 && units() <= most[i] && rows() < longest; ++i) c.csize *= 2;
    if (c.csize == 1) c.warps = 8;
    return c;
}

template <typename T, int L, int R, int CW, class Kernel>
cudaError_t launch(Kernel kernel, const GatedScanArgs &a, int slots, Cut c, cudaStream_t st)
{
    const int slot_bytes = slots * Slot<L, R, CW>::kBytes;   // of a warp
    const int nblocks = ceil_div(a.D, L * kVec<T>);
    const int64_t units = (int64_t)a.N * nblocks;
    const int most = ceil_div(a.T > 0 ? a.T : 1, R * 32 / L);
    const int nwarps = most < c.warps ? most : c.warps;
    if (units * c.csize > 0x7fffffffll) return cudaErrorInvalidValue;
    const int smem = nwarps * slot_bytes + Exchange<T, L>::bytes(nwarps, c.csize);
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e == cudaSuccess && c.csize > 8) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(units * c.csize));
    cfg.blockDim = dim3(32 * (nwarps + (c.csize > 1)));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at = {};
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = c.csize;
    at.val.clusterDim.y = 1;
    at.val.clusterDim.z = 1;
    cfg.attrs = &at;
    cfg.numAttrs = c.csize > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, a, nblocks, c.csize);
}

template <typename T>
int copies_of(const GatedScanArgs &a)
{
    const uintptr_t bases = (uintptr_t)a.x | (uintptr_t)a.g | (uintptr_t)a.out | (uintptr_t)a.h | (uintptr_t)a.dout |
                            (uintptr_t)a.dx | (uintptr_t)a.dg, rows = (uintptr_t)a.D * sizeof(T);
    if (((bases | rows) & 15) == 0) return kWhole;
    if (sizeof(T) == 2 && ((bases | rows) & 3) == 0) return kWords;
    return (bases & 15) == 0 ? kShifted : kElements;
}

template <typename T, bool GATE, int CW>
cudaError_t fwd_cw(const GatedScanArgs &a, cudaStream_t st)
{
    constexpr int R = 8, S = 2, SLOTS = S * 2, CLUSTER_WARPS = 15;
    if constexpr (CW != kElements) {   // that one is there for being right
        const Cut c = cut(a, kVec<T>, R, CLUSTER_WARPS);
        if (c.csize > 1)
            return launch<T, 4, R, CW>(scan_fwd_kernel<T, GATE, CW, 4, R, S, CLUSTER_WARPS, true>, a, SLOTS, c, st);
        if (c.lanes == 4) return launch<T, 4, R, CW>(scan_fwd_kernel<T, GATE, CW, 4, R, S, 8, false>, a, SLOTS, c, st);
        if (c.lanes == 8) return launch<T, 8, R, CW>(scan_fwd_kernel<T, GATE, CW, 8, R, S, 8, false>, a, SLOTS, c, st);
    }
    return launch<T, 16, R, CW>(scan_fwd_kernel<T, GATE, CW, 16, R, S, 8, false>, a, SLOTS, Cut{16, 8, 1}, st);
}

template <typename T, bool GATE, int CW>
cudaError_t bwd_cw(const GatedScanArgs &a, cudaStream_t st)
{
    constexpr int R = GATE ? 4 : 8, S = 2, SLOTS = S * (GATE ? 4 : 3), CLUSTER_WARPS = CW == kShifted ? 10 : 15;
    if constexpr (CW != kElements) {
        const Cut c = cut(a, kVec<T>, R, CLUSTER_WARPS);
        if (c.csize > 1)
            return launch<T, 4, R, CW>(scan_bwd_kernel<T, GATE, CW, 4, R, S, CLUSTER_WARPS, true>, a, SLOTS, c, st);
        // With the gate, 8 rows a thread leave room for one CTA an SM: as many as there are where they are few.
        if (GATE && c.lanes == 4 && (int64_t)a.N * ceil_div(a.D, 4 * kVec<T>) <= 152)
            return launch<T, 4, 8, CW>(scan_bwd_kernel<T, GATE, CW, 4, 8, S, 8, false>, a, SLOTS, c, st);
        if (c.lanes == 4) return launch<T, 4, R, CW>(scan_bwd_kernel<T, GATE, CW, 4, R, S, 8, false>, a, SLOTS, c, st);
        if (c.lanes == 8) return launch<T, 8, R, CW>(scan_bwd_kernel<T, GATE, CW, 8, R, S, 8, false>, a, SLOTS, c, st);
    }
    return launch<T, 16, R, CW>(scan_bwd_kernel<T, GATE, CW, 16, R, S, 8, false>, a, SLOTS, Cut{16, 8, 1}, st);
}

template <typename T, bool GATE>
cudaError_t fwd(const GatedScanArgs &a, cudaStream_t st)
{
    const int c = copies_of<T>(a);
    if constexpr (sizeof(T) == 2)
        if (c == kWords) return fwd_cw<T, GATE, kWords>(a, st);
    return c == kWhole ? fwd_cw<T, GATE, kWhole>(a, st) : c == kShifted ? fwd_cw<T, GATE, kShifted>(a, st)
                                                                        : fwd_cw<T, GATE, kElements>(a, st);
}

template <typename T, bool GATE>
cudaError_t bwd(const GatedScanArgs &a, cudaStream_t st)
{
    const int c = copies_of<T>(a);
    if constexpr (sizeof(T) == 2)
        if (c == kWords) return bwd_cw<T, GATE, kWords>(a, st);
    return c == kWhole ? bwd_cw<T, GATE, kWhole>(a, st) : c == kShifted ? bwd_cw<T, GATE, kShifted>(a, st)
                                                                        : bwd_cw<T, GATE, kElements>(a, st);
}

template <typename T, bool GATE>
cudaError_t step(float *state, const void *x, const void *g, void *out, int64_t n, cudaStream_t st)
{
    const bool wide = n % 8 == 0 && (((uintptr_t)state | (uintptr_t)x | (uintptr_t)g | (uintptr_t)out) & 15) == 0;
    const int64_t blocks = (n + (wide ? 2047 : 255)) / (wide ? 2048 : 256);
    const unsigned grid = (unsigned)(blocks < 152 * 8 ? blocks : 152 * 8);
    if (wide) scan_step_kernel<T, GATE, 8><<<grid, 256, 0, st>>>(state, (const T *)x, (const T *)g, (T *)out, n);
    else scan_step_kernel<T, GATE, 1><<<grid, 256, 0, st>>>(state, (const T *)x, (const T *)g, (T *)out, n);
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
