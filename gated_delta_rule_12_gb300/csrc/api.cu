// api.cu -- the C ABI of libgdn.so (declared in include/gdn.h).
//
// Host-side validation happens first and synchronously; only then is work
// enqueued on the caller's stream.  Nothing here allocates device memory,
// synchronises the device (except gdn_check_device_error) or keeps state
// between calls.
#include <stdint.h>
#include <string.h>

#include "../../include/gdn.h"
#include "common.cuh"
#include "kernels.h"

using namespace gdn;

namespace {

bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }
bool aligned_to(const void *p, unsigned a) { return ((uintptr_t)p & (uintptr_t)(a - 1)) == 0; }

bool chunk_dims_supported(int dk, int dv)
{
    return (dk == 64 || dk == 128 || dk == 256) && dv >= 32 && dv <= 256 && dv % 32 == 0;
}

// the backward kernels are built and tested for dk in {64, 128}
bool bwd_dims_supported(int dk, int dv) { return (dk == 64 || dk == 128 || dk == 256) && dv >= 32 && dv <= 256 && dv % 32 == 0; }

}  // namespace

extern "C" {

const char *gdn_status_string(gdn_status s)
{
    switch (s) {
        case GDN_OK: return "GDN_OK";
        case GDN_ERR_INVALID_ARG: return "GDN_ERR_INVALID_ARG";
        case GDN_ERR_UNSUPPORTED: return "GDN_ERR_UNSUPPORTED";
        case GDN_ERR_WORKSPACE: return "GDN_ERR_WORKSPACE";
        case GDN_ERR_CUDA: return "GDN_ERR_CUDA";
        case GDN_ERR_DEVICE_TIMEOUT: return "GDN_ERR_DEVICE_TIMEOUT";
        case GDN_ERR_RANGE: return "GDN_ERR_RANGE";
    }
    return "GDN_UNKNOWN_STATUS";
}

size_t gdn_chunk_fwd_workspace_size(int32_t B, int32_t T, int32_t H, int32_t dk, int32_t dv,
                                    int32_t num_seqs, gdn_dtype dt)
{
    if (B < 1 || T < 0 || H < 1 || num_seqs < 0) return 0;
    if (dt != GDN_F32 && dt != GDN_BF16) return 0;
    if (!chunk_dims_supported(dk, dv)) return 0;
    const bool varlen = num_seqs > 0;
    if (varlen && B != 1) return 0;
    const int64_t slots = num_slots(B, T, varlen ? num_seqs : B, varlen);
    if (chunk_tc_supported(dt == GDN_BF16 ? 1 : 0, dk, dv, (int64_t)B * T))
        return chunk_tc_workspace_bytes(slots, H);
    return chunk_workspace_layout(slots, H, dk, dv).total;
}

int32_t gdn_chunk_fwd_kernel_count(int32_t B, int32_t T, int32_t H, int32_t dk, int32_t dv,
                                   int32_t num_seqs, gdn_dtype dt)
{
    if (gdn_chunk_fwd_workspace_size(B, T, H, dk, dv, num_seqs, dt) == 0) return 0;
    const int64_t tokens = (int64_t)B * T;
    if (chunk_tc_supported(dt == GDN_BF16 ? 1 : 0, dk, dv, tokens)) return 2;   // UT + recurrence
    return tokens > 0 ? 3 : 1;   // prologue + UT + recurrence, or the state copy alone
}

gdn_status gdn_chunk_fwd(const void *q, const void *k, const void *v, const float *g,
                         const float *beta, const float *init_state, const int32_t *cu_seqlens,
                         int32_t num_seqs, void *out, float *final_state, int32_t B, int32_t T,
                         int32_t H, int32_t dk, int32_t dv, gdn_dtype dt, float scale,
                         int32_t use_qk_l2norm, int32_t chunk_size, void *workspace,
                         size_t workspace_bytes, void *stream)
{
    if (B < 1 || T < 0 || H < 1 || dk < 1 || dv < 1) return GDN_ERR_INVALID_ARG;
    if (dt != GDN_F32 && dt != GDN_BF16) return GDN_ERR_INVALID_ARG;
    if (chunk_size != kChunk) return GDN_ERR_UNSUPPORTED;
    if (!chunk_dims_supported(dk, dv)) return GDN_ERR_UNSUPPORTED;
    const bool varlen = cu_seqlens != nullptr;
    if (varlen && (B != 1 || num_seqs < 1)) return GDN_ERR_INVALID_ARG;
    if (!varlen && num_seqs != 0 && num_seqs != B) return GDN_ERR_INVALID_ARG;
    const int N = varlen ? num_seqs : B;
    const bool have_tokens = (int64_t)B * T > 0;
    if (have_tokens && (!q || !k || !v || !g || !beta || !out)) return GDN_ERR_INVALID_ARG;
    const void *ptrs16[] = {q, k, v, init_state, out, final_state};
    for (const void *p : ptrs16)
        if (p && !aligned16(p)) return GDN_ERR_INVALID_ARG;
    const void *ptrs4[] = {g, beta, cu_seqlens};
    for (const void *p : ptrs4)
        if (p && !aligned_to(p, 4)) return GDN_ERR_INVALID_ARG;
    if (!workspace) return GDN_ERR_WORKSPACE;
    if (((uintptr_t)workspace & 255u) != 0) return GDN_ERR_WORKSPACE;
    const size_t need = gdn_chunk_fwd_workspace_size(B, T, H, dk, dv, varlen ? num_seqs : 0, dt);
    if (need == 0) return GDN_ERR_INVALID_ARG;
    if (workspace_bytes < need) return GDN_ERR_WORKSPACE;

    ChunkArgs a;
    a.q = q; a.k = k; a.v = v; a.g = g; a.beta = beta; a.init_state = init_state;
    a.out = out; a.final_state = final_state;
    a.gm.B = B; a.gm.T = T; a.gm.H = H; a.gm.dk = dk; a.gm.dv = dv; a.gm.N = N;
    a.gm.cu = cu_seqlens;
    a.gm.nct = ceil_div(T, kChunk);
    a.slots = have_tokens ? num_slots(B, T, N, varlen) : 0;
    a.dt = (dt == GDN_BF16) ? 1 : 0;
    a.scale = scale;
    a.l2 = use_qk_l2norm ? 1 : 0;
    a.workspace = workspace;
    cudaStream_t st = (cudaStream_t)stream;
    cudaError_t e = chunk_tc_supported(a.dt, dk, dv, (int64_t)B * T) ? launch_chunk_tc(a, st)
                                                                     : launch_chunk_simt(a, st);
    return e == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

size_t gdn_chunk_bwd_workspace_size(int32_t B, int32_t T, int32_t H, int32_t dk, int32_t dv,
                                    int32_t num_seqs, gdn_dtype dt)
{
    if (B < 1 || T < 0 || H < 1 || num_seqs < 0) return 0;
    if (dt != GDN_F32 && dt != GDN_BF16) return 0;
    if (!bwd_dims_supported(dk, dv)) return 0;
    const bool varlen = num_seqs > 0;
    if (varlen && B != 1) return 0;
    return chunk_bwd_workspace_bytes(num_slots(B, T, varlen ? num_seqs : B, varlen), H, dk, dv);
}

gdn_status gdn_chunk_bwd(const void *q, const void *k, const void *v, const float *g, const float *beta,
                         const float *init_state, const int32_t *cu_seqlens, int32_t num_seqs,
                         const void *dout, const float *dfinal_state,
                         void *dq, void *dk_, void *dv_, float *dg, float *dbeta, float *dinit_state,
                         int32_t B, int32_t T, int32_t H, int32_t dk, int32_t dv, gdn_dtype dt, float scale,
                         int32_t use_qk_l2norm, int32_t chunk_size, void *workspace, size_t workspace_bytes,
                         void *stream)
{
    if (B < 1 || T < 0 || H < 1 || dk < 1 || dv < 1) return GDN_ERR_INVALID_ARG;
    if (dt != GDN_F32 && dt != GDN_BF16) return GDN_ERR_INVALID_ARG;
    if (chunk_size != kChunk) return GDN_ERR_UNSUPPORTED;
    if (!bwd_dims_supported(dk, dv)) return GDN_ERR_UNSUPPORTED;
    const bool varlen = cu_seqlens != nullptr;
    if (varlen && (B != 1 || num_seqs < 1)) return GDN_ERR_INVALID_ARG;
    if (!varlen && num_seqs != 0 && num_seqs != B) return GDN_ERR_INVALID_ARG;
    const int N = varlen ? num_seqs : B;
    const bool have_tokens = (int64_t)B * T > 0;
    if (have_tokens && (!q || !k || !v || !g || !beta || !dout || !dq || !dk_ || !dv_ || !dg || !dbeta))
        return GDN_ERR_INVALID_ARG;
    const void *ptrs16[] = {q, k, v, init_state, dout, dfinal_state, dq, dk_, dv_, dinit_state};
    for (const void *p : ptrs16)
        if (p && !aligned16(p)) return GDN_ERR_INVALID_ARG;
    const void *ptrs4[] = {g, beta, cu_seqlens, dg, dbeta};
    for (const void *p : ptrs4)
        if (p && !aligned_to(p, 4)) return GDN_ERR_INVALID_ARG;
    if (!workspace || ((uintptr_t)workspace & 255u) != 0) return GDN_ERR_WORKSPACE;
    const size_t need = gdn_chunk_bwd_workspace_size(B, T, H, dk, dv, varlen ? num_seqs : 0, dt);
    if (need == 0) return GDN_ERR_INVALID_ARG;
    if (workspace_bytes < need) return GDN_ERR_WORKSPACE;

    BwdArgs a;
    a.q = q; a.k = k; a.v = v; a.dout = dout; a.g = g; a.beta = beta;
    a.init_state = init_state; a.dfinal = dfinal_state;
    a.dq = dq; a.dk = dk_; a.dv = dv_; a.dg = dg; a.dbeta = dbeta; a.dinit = dinit_state;
    a.gm.B = B; a.gm.T = T; a.gm.H = H; a.gm.dk = dk; a.gm.dv = dv; a.gm.N = N;
    a.gm.cu = cu_seqlens;
    a.gm.nct = ceil_div(T, kChunk);
    a.slots = have_tokens ? num_slots(B, T, N, varlen) : 0;
    a.dt = (dt == GDN_BF16) ? 1 : 0;
    a.scale = scale;
    a.l2 = use_qk_l2norm ? 1 : 0;
    a.workspace = workspace;
    cudaError_t e = launch_chunk_bwd(a, (cudaStream_t)stream);
    return e == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

static gdn_status decode_common(float *state, const void *q, const void *k, const void *v, const float *g,
                                const float *beta, void *out, int32_t N, int32_t T, int32_t H, int32_t dk,
                                int32_t dv, gdn_dtype dt, float scale, int32_t use_qk_l2norm, void *stream)
{
    if (N < 0 || T < 0 || H < 1 || dk < 1 || dv < 1) return GDN_ERR_INVALID_ARG;
    if (dt != GDN_F32 && dt != GDN_BF16) return GDN_ERR_INVALID_ARG;
    if (!(dk == 64 || dk == 128 || dk == 256) || dv % 8 != 0) return GDN_ERR_UNSUPPORTED;
    if (N == 0 || T == 0) return GDN_OK;
    if ((int64_t)N * T * H * (dk > dv ? dk : dv) >= ((int64_t)1 << 62)) return GDN_ERR_INVALID_ARG;
    const void *ptrs[] = {state, q, k, v, g, beta, out};
    for (const void *p : ptrs)
        if (!p) return GDN_ERR_INVALID_ARG;
    const unsigned esz = (dt == GDN_BF16) ? 2u : 4u;
    if (!aligned16(state) || !aligned_to(q, esz) || !aligned_to(k, esz) || !aligned_to(v, esz) ||
        !aligned_to(out, esz) || !aligned_to(g, 4) || !aligned_to(beta, 4))
        return GDN_ERR_INVALID_ARG;
    DecodeArgs a;
    a.state = state; a.q = q; a.k = k; a.v = v; a.g = g; a.beta = beta; a.out = out;
    a.N = N; a.H = H; a.dk = dk; a.dv = dv; a.dt = (dt == GDN_BF16) ? 1 : 0;
    a.ntok = T;
    a.scale = scale; a.l2 = use_qk_l2norm ? 1 : 0;
    cudaError_t e = launch_decode(a, (cudaStream_t)stream);
    return e == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

gdn_status gdn_decode_step(float *state, const void *q, const void *k, const void *v,
                           const float *g, const float *beta, void *out, int32_t N, int32_t H,
                           int32_t dk, int32_t dv, gdn_dtype dt, float scale,
                           int32_t use_qk_l2norm, void *stream)
{
    return decode_common(state, q, k, v, g, beta, out, N, 1, H, dk, dv, dt, scale, use_qk_l2norm, stream);
}

gdn_status gdn_decode_multi(float *state, const void *q, const void *k, const void *v,
                            const float *g, const float *beta, void *out, int32_t N, int32_t T,
                            int32_t H, int32_t dk, int32_t dv, gdn_dtype dt, float scale,
                            int32_t use_qk_l2norm, void *stream)
{
    return decode_common(state, q, k, v, g, beta, out, N, T, H, dk, dv, dt, scale, use_qk_l2norm, stream);
}

gdn_status gdn_prologue(const void *xq, const void *xk, const void *xv, const float *wq, const float *wk,
                        const float *wv, const float *a, const float *b, const float *A_log,
                        const float *dt_bias, const void *conv_state_in, void *conv_state_out,
                        const int32_t *cu_seqlens, int32_t num_seqs, void *q, void *k, void *v, float *g,
                        float *beta, int32_t B, int32_t T, int32_t H, int32_t dk, int32_t dv, int32_t K,
                        gdn_dtype dt, void *stream)
{
    if (B < 1 || T < 0 || H < 1 || dk < 1 || dv < 1) return GDN_ERR_INVALID_ARG;
    if (dt != GDN_F32 && dt != GDN_BF16) return GDN_ERR_INVALID_ARG;
    if (K < 1 || K > 4 || dk % 8 != 0 || dv % 8 != 0 || dk > 256 || dv > 256) return GDN_ERR_UNSUPPORTED;
    const bool varlen = cu_seqlens != nullptr;
    if (varlen && (B != 1 || num_seqs < 1)) return GDN_ERR_INVALID_ARG;
    if (!varlen && num_seqs != 0 && num_seqs != B) return GDN_ERR_INVALID_ARG;
    const int N = varlen ? num_seqs : B;
    if ((int64_t)B * T * H >= ((int64_t)1 << 40)) return GDN_ERR_INVALID_ARG;
    const bool have_tokens = (int64_t)B * T > 0;
    if (have_tokens) {
        const void *need[] = {xq, xk, xv, wq, wk, wv, a, b, A_log, dt_bias, q, k, v, g, beta};
        for (const void *p : need)
            if (!p) return GDN_ERR_INVALID_ARG;
    }
    const void *al16[] = {xq, xk, xv, q, k, v, conv_state_in, conv_state_out};
    for (const void *p : al16)
        if (p && !aligned16(p)) return GDN_ERR_INVALID_ARG;
    const void *al4[] = {wq, wk, wv, a, b, A_log, dt_bias, g, beta, cu_seqlens};
    for (const void *p : al4)
        if (p && !aligned_to(p, 4)) return GDN_ERR_INVALID_ARG;
    if (conv_state_in && conv_state_out && K > 1) {   // the two state buffers must not overlap
        const size_t bytes = (size_t)N * (K - 1) * H * (2 * dk + dv) * (dt == GDN_BF16 ? 2 : 4);
        const uintptr_t i0 = (uintptr_t)conv_state_in, o0 = (uintptr_t)conv_state_out;
        if (i0 < o0 + bytes && o0 < i0 + bytes) return GDN_ERR_INVALID_ARG;
    }
    if (!have_tokens && !conv_state_out) return GDN_OK;
    PrologueArgs pa;
    pa.xq = xq; pa.xk = xk; pa.xv = xv; pa.wq = wq; pa.wk = wk; pa.wv = wv;
    pa.a = a; pa.b = b; pa.A_log = A_log; pa.dt_bias = dt_bias;
    pa.state_in = K > 1 ? conv_state_in : nullptr;
    pa.state_out = K > 1 ? conv_state_out : nullptr;
    pa.cu = cu_seqlens;
    pa.q = q; pa.k = k; pa.v = v; pa.g = g; pa.beta = beta;
    pa.B = B; pa.T = T; pa.H = H; pa.dk = dk; pa.dv = dv; pa.N = N; pa.K = K;
    pa.dt = (dt == GDN_BF16) ? 1 : 0;
    cudaError_t e = launch_prologue(pa, (cudaStream_t)stream);
    return e == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

gdn_status gdn_selftest_wait_timeout(void *workspace, uint32_t limit_us, void *stream)
{
    if (!workspace || ((uintptr_t)workspace & 255u) != 0) return GDN_ERR_INVALID_ARG;
    if (limit_us < 1 || limit_us > 1000000u) return GDN_ERR_INVALID_ARG;
    cudaStream_t st = (cudaStream_t)stream;
    if (cudaMemsetAsync(workspace, 0, sizeof(unsigned), st) != cudaSuccess) return GDN_ERR_CUDA;
    cudaError_t e = launch_wait_selftest(reinterpret_cast<unsigned *>(workspace), (uint64_t)limit_us * 1000u, st);
    return e == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

size_t gdn_prologue_chunk_fwd_workspace_size(int32_t B, int32_t T, int32_t H, int32_t dk, int32_t dv,
                                             int32_t num_seqs, gdn_dtype dt)
{
    if (B < 1 || T < 0 || H < 1 || num_seqs < 0) return 0;
    if (dt != GDN_BF16 || !chunk_tc_supported(1, dk, dv, 1)) return 0;
    const bool varlen = num_seqs > 0;
    if (varlen && B != 1) return 0;
    const int64_t slots = (int64_t)B * T > 0 ? num_slots(B, T, varlen ? num_seqs : B, varlen) : 0;
    return chunk_tc_workspace_bytes(slots, H, true);
}

gdn_status gdn_prologue_chunk_fwd(const void *xq, const void *xk, const void *xv, const float *wq,
                                  const float *wk, const float *wv, const float *a, const float *b,
                                  const float *A_log, const float *dt_bias, const void *conv_state_in,
                                  void *conv_state_out, const float *init_state, const int32_t *cu_seqlens,
                                  int32_t num_seqs, void *out, float *final_state, int32_t B, int32_t T,
                                  int32_t H, int32_t dk, int32_t dv, int32_t K, gdn_dtype dt, float scale,
                                  int32_t use_qk_l2norm, int32_t chunk_size, void *workspace,
                                  size_t workspace_bytes, void *stream)
{
    if (B < 1 || T < 0 || H < 1 || dk < 1 || dv < 1) return GDN_ERR_INVALID_ARG;
    if (dt != GDN_F32 && dt != GDN_BF16) return GDN_ERR_INVALID_ARG;
    if (chunk_size != kChunk) return GDN_ERR_UNSUPPORTED;
    if (dt != GDN_BF16 || !chunk_tc_supported(1, dk, dv, 1) || K < 1 || K > 4) return GDN_ERR_UNSUPPORTED;
    const bool varlen = cu_seqlens != nullptr;
    if (varlen && (B != 1 || num_seqs < 1)) return GDN_ERR_INVALID_ARG;
    if (!varlen && num_seqs != 0 && num_seqs != B) return GDN_ERR_INVALID_ARG;
    const int N = varlen ? num_seqs : B;
    const int64_t tokens = (int64_t)B * T;
    if (tokens >= ((int64_t)1 << 31)) return GDN_ERR_INVALID_ARG;
    const bool have_tokens = tokens > 0;
    if (have_tokens) {
        const void *need[] = {xq, xk, xv, wq, wk, wv, a, b, A_log, dt_bias, out};
        for (const void *p : need)
            if (!p) return GDN_ERR_INVALID_ARG;
    }
    const void *al16[] = {xq, xk, xv, out, init_state, final_state, conv_state_in, conv_state_out};
    for (const void *p : al16)
        if (p && !aligned16(p)) return GDN_ERR_INVALID_ARG;
    const void *al4[] = {wq, wk, wv, a, b, A_log, dt_bias, cu_seqlens};
    for (const void *p : al4)
        if (p && !aligned_to(p, 4)) return GDN_ERR_INVALID_ARG;
    if (conv_state_in && conv_state_out && K > 1) {   // the two state buffers must not overlap
        const size_t bytes = (size_t)N * (K - 1) * H * (2 * dk + dv) * 2;
        const uintptr_t i0 = (uintptr_t)conv_state_in, o0 = (uintptr_t)conv_state_out;
        if (i0 < o0 + bytes && o0 < i0 + bytes) return GDN_ERR_INVALID_ARG;
    }
    if (!workspace || ((uintptr_t)workspace & 255u) != 0) return GDN_ERR_WORKSPACE;
    const size_t need = gdn_prologue_chunk_fwd_workspace_size(B, T, H, dk, dv, varlen ? num_seqs : 0, dt);
    if (need == 0) return GDN_ERR_INVALID_ARG;
    if (workspace_bytes < need) return GDN_ERR_WORKSPACE;

    PrologueArgs pa;
    pa.xq = xq; pa.xk = xk; pa.xv = xv; pa.wq = wq; pa.wk = wk; pa.wv = wv;
    pa.a = a; pa.b = b; pa.A_log = A_log; pa.dt_bias = dt_bias;
    pa.state_in = K > 1 ? conv_state_in : nullptr;
    pa.state_out = K > 1 ? conv_state_out : nullptr;
    pa.cu = cu_seqlens;
    pa.q = nullptr; pa.k = nullptr; pa.v = nullptr; pa.g = nullptr; pa.beta = nullptr;
    pa.B = B; pa.T = T; pa.H = H; pa.dk = dk; pa.dv = dv; pa.N = N; pa.K = K;
    pa.dt = 1;
    ChunkArgs ca;
    ca.q = nullptr; ca.k = nullptr; ca.v = nullptr; ca.g = nullptr; ca.beta = nullptr;
    ca.init_state = init_state; ca.out = out; ca.final_state = final_state;
    ca.gm.B = B; ca.gm.T = T; ca.gm.H = H; ca.gm.dk = dk; ca.gm.dv = dv; ca.gm.N = N;
    ca.gm.cu = cu_seqlens;
    ca.gm.nct = ceil_div(T, kChunk);
    ca.slots = have_tokens ? num_slots(B, T, N, varlen) : 0;
    ca.dt = 1;
    ca.scale = scale;
    ca.l2 = use_qk_l2norm ? 1 : 0;
    ca.workspace = workspace;
    cudaStream_t st = (cudaStream_t)stream;
    cudaError_t e;
    if (!have_tokens) {
        // nothing to transform: the states pass through (the prologue kernel carries the
        // convolution state of empty sequences; the CUDA-core path copies init to final)
        e = pa.state_out ? launch_prologue(pa, st) : cudaSuccess;
        if (e == cudaSuccess) e = launch_chunk_simt(ca, st);
    } else {
        ca.fuse = &pa;
        e = launch_chunk_tc(ca, st);
    }
    return e == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

static gdn_status scan_geometry(GatedScanArgs &a, const int32_t *cu_seqlens, int32_t num_seqs, int32_t B, int32_t T,
                                int32_t D, gdn_dtype dt, int32_t input_gate)
{
    if (B < 1 || T < 0 || D < 1) return GDN_ERR_INVALID_ARG;
    if (dt != GDN_F32 && dt != GDN_BF16) return GDN_ERR_INVALID_ARG;
    if (cu_seqlens ? (B != 1 || num_seqs < 1) : (num_seqs != 0 && num_seqs != B)) return GDN_ERR_INVALID_ARG;
    if (!aligned_to(cu_seqlens, 4)) return GDN_ERR_INVALID_ARG;
    a = GatedScanArgs();
    a.cu = cu_seqlens;
    a.N = cu_seqlens ? num_seqs : B;
    a.T = T; a.D = D;
    a.dt = (dt == GDN_BF16) ? 1 : 0;
    a.input_gate = input_gate ? 1 : 0;
    return GDN_OK;
}

gdn_status gdn_gated_scan_fwd(const void *x, const void *g, const float *init_state, const int32_t *cu_seqlens,
                              int32_t num_seqs, void *out, float *final_state, int32_t B, int32_t T, int32_t D,
                              gdn_dtype dt, int32_t input_gate, void *stream)
{
    GatedScanArgs a;
    const gdn_status s = scan_geometry(a, cu_seqlens, num_seqs, B, T, D, dt, input_gate);
    if (s != GDN_OK) return s;
    const bool have_tokens = (int64_t)B * T > 0;
    if (have_tokens && (!x || !g || !out)) return GDN_ERR_INVALID_ARG;
    const unsigned esz = (dt == GDN_BF16) ? 2u : 4u;
    if (!aligned_to(x, esz) || !aligned_to(g, esz) || !aligned_to(out, esz) || !aligned_to(init_state, 4) ||
        !aligned_to(final_state, 4))
        return GDN_ERR_INVALID_ARG;
    if (!have_tokens && !final_state) return GDN_OK;
    a.x = x; a.g = g; a.init_state = init_state; a.out = out; a.final_state = final_state;
    return launch_gated_scan_fwd(a, (cudaStream_t)stream) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

gdn_status gdn_gated_scan_bwd(const void *x, const void *g, const void *out, const void *dout,
                              const float *init_state, const float *dfinal_state, const int32_t *cu_seqlens,
                              int32_t num_seqs, void *dx, void *dg, float *dinit_state, int32_t B, int32_t T,
                              int32_t D, gdn_dtype dt, int32_t input_gate, void *stream)
{
    GatedScanArgs a;
    const gdn_status s = scan_geometry(a, cu_seqlens, num_seqs, B, T, D, dt, input_gate);
    if (s != GDN_OK) return s;
    const bool have_tokens = (int64_t)B * T > 0;
    if (have_tokens && ((input_gate && !x) || !g || !out || !dout || !dx || !dg)) return GDN_ERR_INVALID_ARG;
    const unsigned esz = (dt == GDN_BF16) ? 2u : 4u;
    const void *elems[] = {x, g, out, dout, dx, dg};
    for (const void *p : elems)
        if (!aligned_to(p, esz)) return GDN_ERR_INVALID_ARG;
    if (!aligned_to(init_state, 4) || !aligned_to(dfinal_state, 4) || !aligned_to(dinit_state, 4))
        return GDN_ERR_INVALID_ARG;
    if (!have_tokens && !dinit_state) return GDN_OK;
    a.x = x; a.g = g; a.h = out; a.dout = dout; a.init_state = init_state; a.dfinal = dfinal_state;
    a.dx = dx; a.dg = dg; a.dinit = dinit_state;
    return launch_gated_scan_bwd(a, (cudaStream_t)stream) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

gdn_status gdn_gated_scan_step(float *state, const void *x, const void *g, void *out, int32_t N, int32_t D,
                               gdn_dtype dt, int32_t input_gate, void *stream)
{
    if (N < 0 || D < 1) return GDN_ERR_INVALID_ARG;
    if (dt != GDN_F32 && dt != GDN_BF16) return GDN_ERR_INVALID_ARG;
    if (N == 0) return GDN_OK;
    const unsigned esz = (dt == GDN_BF16) ? 2u : 4u;
    if (!state || !x || !g || !out || !aligned_to(state, 4) || !aligned_to(x, esz) || !aligned_to(g, esz) ||
        !aligned_to(out, esz))
        return GDN_ERR_INVALID_ARG;
    const cudaError_t e = launch_gated_scan_step(state, x, g, out, (int64_t)N * D, (dt == GDN_BF16) ? 1 : 0,
                                                 input_gate ? 1 : 0, (cudaStream_t)stream);
    return e == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

gdn_status gdn_layer_norm_fwd(const void *x, const float *weight, const float *bias, void *out, float *mean,
                              float *rstd, int64_t rows, int32_t D, gdn_dtype dt, float eps, void *stream)
{
    if (rows < 0 || D < 1 || !(eps >= 0.f)) return GDN_ERR_INVALID_ARG;
    if (dt != GDN_F32 && dt != GDN_BF16) return GDN_ERR_INVALID_ARG;
    if (rows > ((int64_t)1 << 48) / D) return GDN_ERR_INVALID_ARG;
    if (rows == 0) return GDN_OK;
    const unsigned esz = (dt == GDN_BF16) ? 2u : 4u;
    if (!x || !out || !aligned_to(x, esz) || !aligned_to(out, esz)) return GDN_ERR_INVALID_ARG;
    const void *ptrs4[] = {weight, bias, mean, rstd};
    for (const void *p : ptrs4)
        if (!aligned_to(p, 4)) return GDN_ERR_INVALID_ARG;
    LayerNormArgs a = LayerNormArgs();
    a.x = x; a.weight = weight; a.bias = bias; a.out = out; a.mean = mean; a.rstd = rstd;
    a.rows = rows; a.D = D; a.dt = (dt == GDN_BF16) ? 1 : 0; a.eps = eps;
    return launch_layer_norm_fwd(a, (cudaStream_t)stream) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

size_t gdn_layer_norm_bwd_workspace_size(int64_t rows, int32_t D, gdn_dtype dt)
{
    if (rows < 0 || D < 1 || (dt != GDN_F32 && dt != GDN_BF16) || rows > ((int64_t)1 << 48) / D) return 0;
    return layer_norm_bwd_workspace_bytes(rows, D, (dt == GDN_BF16) ? 1 : 0);
}

gdn_status gdn_layer_norm_bwd(const void *dout, const void *x, const float *mean, const float *rstd,
                              const float *weight, void *dx, float *dweight, float *dbias, int64_t rows, int32_t D,
                              gdn_dtype dt, void *workspace, size_t workspace_bytes, void *stream)
{
    if (rows < 0 || D < 1) return GDN_ERR_INVALID_ARG;
    if (dt != GDN_F32 && dt != GDN_BF16) return GDN_ERR_INVALID_ARG;
    if (rows > ((int64_t)1 << 48) / D) return GDN_ERR_INVALID_ARG;
    const unsigned esz = (dt == GDN_BF16) ? 2u : 4u;
    if (rows > 0 && (!dout || !x || !mean || !rstd)) return GDN_ERR_INVALID_ARG;
    if (!aligned_to(dout, esz) || !aligned_to(x, esz) || !aligned_to(dx, esz)) return GDN_ERR_INVALID_ARG;
    const void *ptrs4[] = {mean, rstd, weight, dweight, dbias};
    for (const void *p : ptrs4)
        if (!aligned_to(p, 4)) return GDN_ERR_INVALID_ARG;
    if (!workspace || ((uintptr_t)workspace & 255u) != 0) return GDN_ERR_WORKSPACE;
    if (workspace_bytes < gdn_layer_norm_bwd_workspace_size(rows, D, dt)) return GDN_ERR_WORKSPACE;
    LayerNormArgs a = LayerNormArgs();
    a.dout = dout; a.x = x; a.mean = const_cast<float *>(mean); a.rstd = const_cast<float *>(rstd);
    a.weight = weight; a.dx = dx; a.dweight = dweight; a.dbias = dbias;
    a.rows = rows; a.D = D; a.dt = (dt == GDN_BF16) ? 1 : 0;
    a.workspace = workspace;
    return launch_layer_norm_bwd(a, (cudaStream_t)stream) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

static gdn_status rms_args(RmsNormArgs &a, const void *x, const void *residual, const float *weight, void *out,
                           void *residual_out, int64_t rows, int32_t D, gdn_dtype dt, float eps, unsigned out_size)
{
    if (rows < 0 || D < 1 || !(eps >= 0.f)) return GDN_ERR_INVALID_ARG;
    if (dt != GDN_F32 && dt != GDN_BF16) return GDN_ERR_INVALID_ARG;
    if (rows > ((int64_t)1 << 48) / D) return GDN_ERR_INVALID_ARG;
    if (!residual != !residual_out && rows > 0) return GDN_ERR_INVALID_ARG;
    const unsigned esz = (dt == GDN_BF16) ? 2u : 4u;
    if (rows > 0 && (!x || !out)) return GDN_ERR_INVALID_ARG;
    if (!aligned_to(x, esz) || !aligned_to(residual, esz) || !aligned_to(residual_out, esz) || !aligned_to(out, out_size) ||
        !aligned_to(weight, 4))
        return GDN_ERR_INVALID_ARG;
    a = RmsNormArgs();
    a.x = x; a.residual = residual; a.weight = weight; a.out = out; a.residual_out = residual_out;
    a.rows = rows; a.D = D; a.dt = (dt == GDN_BF16) ? 1 : 0; a.eps = eps;
    return GDN_OK;
}

gdn_status gdn_rms_norm_fwd(const void *x, const void *residual, const float *weight, void *out, void *residual_out,
                            float *rstd, int64_t rows, int32_t D, gdn_dtype dt, float eps, void *stream)
{
    RmsNormArgs a;
    const gdn_status s = rms_args(a, x, residual, weight, out, residual_out, rows, D, dt, eps, (dt == GDN_BF16) ? 2u : 4u);
    if (s != GDN_OK) return s;
    if (!aligned_to(rstd, 4) || (rows > 0 && out == residual_out)) return GDN_ERR_INVALID_ARG;
    if (rows == 0) return GDN_OK;
    a.rstd = rstd;
    return launch_rms_norm_fwd(a, (cudaStream_t)stream) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

gdn_status gdn_rms_norm_fp8(const void *x, const void *residual, const float *weight, void *q, float *scales,
                            void *residual_out, int64_t rows, int32_t D, gdn_dtype dt, float eps, void *stream)
{
    RmsNormArgs a;
    const gdn_status s = rms_args(a, x, residual, weight, q, residual_out, rows, D, dt, eps, 1u);
    if (s != GDN_OK) return s;
    if ((rows > 0 && !scales) || !aligned_to(scales, 4)) return GDN_ERR_INVALID_ARG;
    if (rows == 0) return GDN_OK;
    a.scales = scales;
    return launch_rms_norm_fwd(a, (cudaStream_t)stream) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

size_t gdn_rms_norm_bwd_workspace_size(int64_t rows, int32_t D, gdn_dtype dt)
{
    if (rows < 0 || D < 1 || (dt != GDN_F32 && dt != GDN_BF16) || rows > ((int64_t)1 << 48) / D) return 0;
    return rms_norm_bwd_workspace_bytes(D);
}

gdn_status gdn_rms_norm_bwd(const void *dout, const void *x, const float *rstd, const float *weight, const void *dresidual,
                            void *dx, float *dweight, int64_t rows, int32_t D, gdn_dtype dt, void *workspace,
                            size_t workspace_bytes, void *stream)
{
    if (rows < 0 || D < 1) return GDN_ERR_INVALID_ARG;
    if (dt != GDN_F32 && dt != GDN_BF16) return GDN_ERR_INVALID_ARG;
    if (rows > ((int64_t)1 << 48) / D) return GDN_ERR_INVALID_ARG;
    const unsigned esz = (dt == GDN_BF16) ? 2u : 4u;
    if (rows > 0 && (!dout || !x || !rstd)) return GDN_ERR_INVALID_ARG;
    if (!aligned_to(dout, esz) || !aligned_to(x, esz) || !aligned_to(dresidual, esz) || !aligned_to(dx, esz) ||
        !aligned_to(rstd, 4) || !aligned_to(weight, 4) || !aligned_to(dweight, 4))
        return GDN_ERR_INVALID_ARG;
    if (!workspace || ((uintptr_t)workspace & 255u) != 0) return GDN_ERR_WORKSPACE;
    if (workspace_bytes < gdn_rms_norm_bwd_workspace_size(rows, D, dt)) return GDN_ERR_WORKSPACE;
    if (!dx && !dweight) return GDN_OK;
    if (rows == 0) {
        if (!dweight) return GDN_OK;
        return cudaMemsetAsync(dweight, 0, (size_t)D * 4, (cudaStream_t)stream) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
    }
    RmsNormArgs a = RmsNormArgs();
    a.dout = dout; a.x = x; a.rstd = const_cast<float *>(rstd); a.weight = weight; a.dresidual = dx ? dresidual : nullptr;
    a.dx = dx; a.dweight = dweight;
    a.rows = rows; a.D = D; a.dt = (dt == GDN_BF16) ? 1 : 0;
    a.workspace = workspace;
    return launch_rms_norm_bwd(a, (cudaStream_t)stream) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

gdn_status gdn_fp8_quantize(const void *x, void *q, float *scales, int64_t rows, int32_t D, int32_t block_rows,
                            gdn_dtype dt, void *stream)
{
    if (rows < 0 || D < 1 || (block_rows != 1 && block_rows != kFp8Block)) return GDN_ERR_INVALID_ARG;
    if (dt != GDN_F32 && dt != GDN_BF16) return GDN_ERR_INVALID_ARG;
    if (rows > ((int64_t)1 << 48) / D) return GDN_ERR_INVALID_ARG;
    if (rows > 0 && (!x || !q || !scales)) return GDN_ERR_INVALID_ARG;
    if (!aligned_to(x, (dt == GDN_BF16) ? 2u : 4u) || !aligned_to(scales, 4)) return GDN_ERR_INVALID_ARG;
    if (block_rows > 1 && (rows + kFp8Block - 1) / kFp8Block * ceil_div(D, kFp8Block) > INT32_MAX) return GDN_ERR_UNSUPPORTED;
    if (rows == 0) return GDN_OK;
    Fp8QuantArgs a = Fp8QuantArgs();
    a.x = x; a.q = (unsigned char *)q; a.scales = scales;
    a.rows = rows; a.D = D; a.dt = (dt == GDN_BF16) ? 1 : 0; a.block_rows = block_rows;
    return launch_fp8_quantize(a, (cudaStream_t)stream) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

// launch grids and tile counts stay within 32 bits
static bool fp8_size_supported(int32_t M, int32_t N, int32_t K)
{
    return M <= (1 << 23) && N <= (1 << 23) && (int64_t)M * N <= (int64_t)1 << 42 && K <= (1 << 20);
}

size_t gdn_fp8_linear_workspace_size(int32_t M, int32_t N, int32_t K)
{
    if (M < 0 || N < 1 || K < 1 || !fp8_size_supported(M, N, K)) return 0;
    return fp8_linear_workspace_bytes(M, N, K);
}

static gdn_status fp8_args(Fp8LinearArgs &a, const void *x, const float *x_scales, const void *w, const float *w_scales,
                           void *out, int32_t M, int32_t N, int32_t K, void *workspace, size_t workspace_bytes)
{
    if (M < 0 || N < 1 || K < 1) return GDN_ERR_INVALID_ARG;
    if (!fp8_size_supported(M, N, K)) return GDN_ERR_UNSUPPORTED;
    if (M > 0 && (!x || !x_scales || !out)) return GDN_ERR_INVALID_ARG;
    if (!w || !w_scales || !aligned_to(x_scales, 4) || !aligned_to(w_scales, 4) || !aligned_to(out, 2)) return GDN_ERR_INVALID_ARG;
    if (!workspace || ((uintptr_t)workspace & 255u) != 0) return GDN_ERR_WORKSPACE;
    if (workspace_bytes < gdn_fp8_linear_workspace_size(M, N, K)) return GDN_ERR_WORKSPACE;
    a = Fp8LinearArgs();
    a.x = (const unsigned char *)x; a.w = (const unsigned char *)w; a.xs = x_scales; a.ws = w_scales; a.out = out;
    a.M = M; a.N = N; a.K = K;
    a.workspace = workspace;
    return GDN_OK;
}

gdn_status gdn_fp8_linear(const void *x, const float *x_scales, const void *w, const float *w_scales, void *out, int32_t M,
                          int32_t N, int32_t K, void *workspace, size_t workspace_bytes, void *stream)
{
    Fp8LinearArgs a;
    const gdn_status s = fp8_args(a, x, x_scales, w, w_scales, out, M, N, K, workspace, workspace_bytes);
    if (s != GDN_OK || M == 0) return s;
    return launch_fp8_linear(a, (cudaStream_t)stream) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

gdn_status gdn_selftest_fp8_linear_timeout(uint32_t limit_us, const void *x, const float *x_scales, const void *w,
                                           const float *w_scales, void *out, int32_t M, int32_t N, int32_t K,
                                           void *workspace, size_t workspace_bytes, void *stream)
{
    Fp8LinearArgs a;
    if (limit_us < 1 || limit_us > 1000000u) return GDN_ERR_INVALID_ARG;
    const gdn_status s = fp8_args(a, x, x_scales, w, w_scales, out, M, N, K, workspace, workspace_bytes);
    if (s != GDN_OK) return s;
    if (M < 1) return GDN_ERR_INVALID_ARG;
    if (!fp8_linear_tc_supported(a)) return GDN_ERR_UNSUPPORTED;
    return launch_fp8_linear_tc(a, (cudaStream_t)stream, (uint64_t)limit_us * 1000u) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

// launch grids and tile counts stay within 32 bits
static bool ce_size_supported(int32_t N, int32_t V)
{
    return N <= (1 << 23) && V <= (1 << 30) && (int64_t)N * V <= (int64_t)1 << 45;
}

size_t gdn_linear_cross_entropy_workspace_size(int32_t N, int32_t D, int32_t V, gdn_dtype dt, int32_t backward)
{
    if (N < 0 || D < 1 || V < 1 || (dt != GDN_F32 && dt != GDN_BF16) || !ce_size_supported(N, V)) return 0;
    return linear_ce_workspace_bytes(N, D, V, (dt == GDN_BF16) ? 1 : 0, backward != 0);
}

static gdn_status ce_args(LinearCeArgs &a, const void *h, const void *weight, const int32_t *targets, int32_t N,
                          int32_t D, int32_t V, gdn_dtype dt, bool backward, void *workspace, size_t workspace_bytes)
{
    if (N < 0 || D < 1 || V < 1) return GDN_ERR_INVALID_ARG;
    if (dt != GDN_F32 && dt != GDN_BF16) return GDN_ERR_INVALID_ARG;
    if (N > 0 && (!h || !targets)) return GDN_ERR_INVALID_ARG;
    if (!ce_size_supported(N, V)) return GDN_ERR_UNSUPPORTED;
    if (!weight) return GDN_ERR_INVALID_ARG;
    if (!aligned16(h) || !aligned16(weight) || !aligned_to(targets, 4)) return GDN_ERR_INVALID_ARG;
    if (!workspace || ((uintptr_t)workspace & 255u) != 0) return GDN_ERR_WORKSPACE;
    if (workspace_bytes < gdn_linear_cross_entropy_workspace_size(N, D, V, dt, backward)) return GDN_ERR_WORKSPACE;
    a = LinearCeArgs();
    a.h = h; a.w = weight; a.targets = targets;
    a.N = N; a.D = D; a.V = V; a.dt = (dt == GDN_BF16) ? 1 : 0;
    a.workspace = workspace;
    return GDN_OK;
}

gdn_status gdn_linear_cross_entropy_fwd(const void *h, const void *weight, const int32_t *targets, float *loss,
                                        float *lse, int32_t N, int32_t D, int32_t V, gdn_dtype dt, void *workspace,
                                        size_t workspace_bytes, void *stream)
{
    LinearCeArgs a;
    const gdn_status s = ce_args(a, h, weight, targets, N, D, V, dt, false, workspace, workspace_bytes);
    if (s != GDN_OK) return s;
    if ((N > 0 && !loss) || !aligned_to(loss, 4) || !aligned_to(lse, 4)) return GDN_ERR_INVALID_ARG;
    if (N == 0) return GDN_OK;
    a.loss = loss; a.lse = lse;
    return launch_linear_ce_fwd(a, (cudaStream_t)stream) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

gdn_status gdn_linear_cross_entropy_bwd(const void *h, const void *weight, const int32_t *targets, const float *lse,
                                        const float *dloss, void *dh, void *dweight, int32_t N, int32_t D, int32_t V,
                                        gdn_dtype dt, void *workspace, size_t workspace_bytes, void *stream)
{
    LinearCeArgs a;
    const gdn_status s = ce_args(a, h, weight, targets, N, D, V, dt, true, workspace, workspace_bytes);
    if (s != GDN_OK) return s;
    if ((N > 0 && (!lse || !dloss)) || !aligned_to(lse, 4) || !aligned_to(dloss, 4) || !aligned16(dh) ||
        !aligned16(dweight))
        return GDN_ERR_INVALID_ARG;
    if (!dh && !dweight) return GDN_OK;
    if (N == 0) {
        if (!dweight) return GDN_OK;
        const size_t bytes = (size_t)V * D * (dt == GDN_BF16 ? 2 : 4);
        return cudaMemsetAsync(dweight, 0, bytes, (cudaStream_t)stream) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
    }
    a.lse_in = lse; a.dloss = dloss; a.dh = dh; a.dw = dweight;
    return launch_linear_ce_bwd(a, (cudaStream_t)stream) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

size_t gdn_linear_log_probs_workspace_size(int32_t N, int32_t D, int32_t V, int32_t top_k, gdn_dtype dt, int32_t backward)
{
    if (N < 0 || D < 1 || V < 1 || top_k < 0 || top_k > GDN_MOST_TOP || top_k > V || (dt != GDN_F32 && dt != GDN_BF16) ||
        !ce_size_supported(N, V))
        return 0;
    return linear_ce_workspace_bytes(N, D, V, (dt == GDN_BF16) ? 1 : 0, backward != 0, backward ? -1 : top_k);
}

gdn_status gdn_linear_log_probs_fwd(const void *h, const void *weight, const int32_t *targets, float *logp, float *entropy,
                                    float *lse, int32_t *top_ids, float *top_logps, int32_t N, int32_t D, int32_t V,
                                    int32_t top_k, gdn_dtype dt, void *workspace, size_t workspace_bytes, void *stream)
{
    LinearCeArgs a;
    if (top_k < 0 || top_k > GDN_MOST_TOP || top_k > V) return GDN_ERR_INVALID_ARG;
    const gdn_status s = ce_args(a, h, weight, targets, N, D, V, dt, false, workspace, SIZE_MAX);
    if (s != GDN_OK) return s;
    if (workspace_bytes < gdn_linear_log_probs_workspace_size(N, D, V, top_k, dt, 0)) return GDN_ERR_WORKSPACE;
    if (N > 0 && (!logp || !entropy || (top_k > 0 && (!top_ids || !top_logps)))) return GDN_ERR_INVALID_ARG;
    const void *ptrs4[] = {logp, entropy, lse, top_ids, top_logps};
    for (const void *p : ptrs4)
        if (!aligned_to(p, 4)) return GDN_ERR_INVALID_ARG;
    if (N == 0) return GDN_OK;
    const LogProbs out = {logp, entropy, lse, top_ids, top_logps, top_k};
    return launch_linear_ce_fwd(a, (cudaStream_t)stream, &out) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

gdn_status gdn_linear_log_probs_bwd(const void *h, const void *weight, const int32_t *targets, const float *lse,
                                    const float *entropy, const float *dlogp, const float *dentropy, void *dh,
                                    void *dweight, int32_t N, int32_t D, int32_t V, gdn_dtype dt, void *workspace,
                                    size_t workspace_bytes, void *stream)
{
    LinearCeArgs a;
    const gdn_status s = ce_args(a, h, weight, targets, N, D, V, dt, true, workspace, workspace_bytes);
    if (s != GDN_OK) return s;
    if (N > 0 && (!lse || !dlogp || (dentropy && !entropy))) return GDN_ERR_INVALID_ARG;
    if (!aligned_to(lse, 4) || !aligned_to(entropy, 4) || !aligned_to(dlogp, 4) || !aligned_to(dentropy, 4) ||
        !aligned16(dh) || !aligned16(dweight))
        return GDN_ERR_INVALID_ARG;
    if (!dh && !dweight) return GDN_OK;
    if (N == 0) {
        if (!dweight) return GDN_OK;
        const size_t bytes = (size_t)V * D * (dt == GDN_BF16 ? 2 : 4);
        return cudaMemsetAsync(dweight, 0, bytes, (cudaStream_t)stream) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
    }
    a.lse_in = lse; a.dloss = dlogp; a.dh = dh; a.dw = dweight;
    return launch_linear_ce_bwd(a, (cudaStream_t)stream, {dentropy, entropy, -1.f}) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

gdn_status gdn_selftest_linear_log_probs_timeout(uint32_t limit_us, const void *h, const void *weight,
                                                 const int32_t *targets, float *logp, float *entropy, int32_t *top_ids,
                                                 float *top_logps, int32_t N, int32_t D, int32_t V, int32_t top_k,
                                                 void *workspace, size_t workspace_bytes, void *stream)
{
    LinearCeArgs a;
    if (limit_us < 1 || limit_us > 1000000u || top_k < 0 || top_k > GDN_MOST_TOP || top_k > V) return GDN_ERR_INVALID_ARG;
    const gdn_status s = ce_args(a, h, weight, targets, N, D, V, GDN_BF16, false, workspace, SIZE_MAX);
    if (s != GDN_OK) return s;
    if (!linear_ce_tc_supported(1, D)) return GDN_ERR_UNSUPPORTED;
    if (workspace_bytes < gdn_linear_log_probs_workspace_size(N, D, V, top_k, GDN_BF16, 0)) return GDN_ERR_WORKSPACE;
    if (N < 1 || !logp || !entropy || (top_k > 0 && (!top_ids || !top_logps))) return GDN_ERR_INVALID_ARG;
    const void *ptrs4[] = {logp, entropy, top_ids, top_logps};
    for (const void *p : ptrs4)
        if (!aligned_to(p, 4)) return GDN_ERR_INVALID_ARG;
    const LogProbs out = {logp, entropy, nullptr, top_ids, top_logps, top_k};
    CeStall stall;
    stall.step = 3;
    stall.limit_ns = (uint64_t)limit_us * 1000u;
    return launch_linear_ce_tc_fwd(a, (cudaStream_t)stream, &out, stall) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

gdn_status gdn_selftest_linear_cross_entropy_timeout(int32_t step, uint32_t limit_us, const void *h, const void *weight,
                                                     const int32_t *targets, const float *lse, const float *dloss,
                                                     void *out0, void *out1, int32_t N, int32_t D, int32_t V,
                                                     void *workspace, size_t workspace_bytes, void *stream)
{
    LinearCeArgs a;
    if (step < 0 || step > 2 || limit_us < 1 || limit_us > 1000000u) return GDN_ERR_INVALID_ARG;
    const gdn_status s = ce_args(a, h, weight, targets, N, D, V, GDN_BF16, step > 0, workspace, workspace_bytes);
    if (s != GDN_OK) return s;
    if (!linear_ce_tc_supported(1, D)) return GDN_ERR_UNSUPPORTED;
    if (N < 1 || !out0 || !aligned16(out0) || !aligned16(out1)) return GDN_ERR_INVALID_ARG;
    CeStall stall;
    stall.step = step;
    stall.limit_ns = (uint64_t)limit_us * 1000u;
    cudaError_t e;
    if (step == 0) {
        a.loss = (float *)out0; a.lse = (float *)out1;
        e = launch_linear_ce_tc_fwd(a, (cudaStream_t)stream, nullptr, stall);
    } else {
        if (!lse || !dloss || !aligned_to(lse, 4) || !aligned_to(dloss, 4)) return GDN_ERR_INVALID_ARG;
        a.lse_in = lse; a.dloss = dloss; a.dh = out0; a.dw = out1;
        e = launch_linear_ce_tc_bwd(a, (cudaStream_t)stream, LogProbsGrad(), stall);
    }
    return e == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

gdn_status gdn_check_device_error(void *workspace, void *stream)
{
    if (!workspace || ((uintptr_t)workspace & 255u) != 0) return GDN_ERR_INVALID_ARG;
    cudaStream_t st = (cudaStream_t)stream;
    unsigned word = 0;
    if (cudaMemcpyAsync(&word, workspace, sizeof(word), cudaMemcpyDeviceToHost, st) != cudaSuccess)
        return GDN_ERR_CUDA;
    if (cudaStreamSynchronize(st) != cudaSuccess) return GDN_ERR_CUDA;
    if (word == kDevErrNone) return GDN_OK;
    if (cudaMemsetAsync(workspace, 0, sizeof(word), st) != cudaSuccess) return GDN_ERR_CUDA;
    if (cudaStreamSynchronize(st) != cudaSuccess) return GDN_ERR_CUDA;
    if (word == kDevErrTimeout) return GDN_ERR_DEVICE_TIMEOUT;
    if (word == kDevErrRange) return GDN_ERR_RANGE;
    return GDN_ERR_CUDA;
}

}  // extern "C"
