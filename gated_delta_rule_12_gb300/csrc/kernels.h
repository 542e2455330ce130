// kernels.h -- internal launcher interface between the C ABI (api.cu) and the
// kernel translation units.  Not part of the public ABI.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"

namespace gdn {

struct PrologueArgs;

struct ChunkArgs {
    const void *q, *k, *v;
    const float *g, *beta, *init_state;
    void *out;
    float *final_state;
    Geometry gm;
    int64_t slots;
    int dt;          // 0 = fp32, 1 = bf16
    float scale;
    int l2;
    void *workspace;
    const PrologueArgs *fuse = nullptr;   // non-null: q, k, v, g, beta are made from these projections
    // Tensor-core path, for the backward pass: chunk-local blocks at blocks + (slot * H + h) * block_stride
    // (instead of after the workspace header), and the chunk-start states and V_new saved (see RcParams).
    void *blocks = nullptr;
    size_t block_stride = 0;
    float *save_s = nullptr, *save_vn = nullptr;
    int64_t save_stride = 0;
};

struct DecodeArgs {
    float *state;
    const void *q, *k, *v;
    const float *g, *beta;
    void *out;
    int N, H, dk, dv, dt;
    int ntok;        // tokens per sequence in this call (1 = single step)
    float scale;
    int l2;
};

struct PrologueArgs {
    const void *xq, *xk, *xv;                 // raw projections [B, T, H, dk|dk|dv], dtype dt
    const float *wq, *wk, *wv;                // convolution filters [H, d, K]
    const float *a, *b, *A_log, *dt_bias;     // gate projections [B, T, H]; per-head parameters [H]
    const void *state_in;                     // [N, K-1, H, 2 dk + dv] dtype dt, or null
    void *state_out;                          // same layout, or null
    const int32_t *cu;                        // [N + 1] or null
    void *q, *k, *v;                          // outputs [B, T, H, dk|dk|dv], dtype dt
    float *g, *beta;                          // outputs [B, T, H]
    int B, T, H, dk, dv, N, K, dt;
};

struct BwdArgs {
    const void *q, *k, *v, *dout;            // dtype dt
    const float *g, *beta, *init_state, *dfinal;
    void *dq, *dk, *dv;                      // dtype dt
    float *dg, *dbeta, *dinit;
    Geometry gm;
    int64_t slots;
    int dt;
    float scale;
    int l2;
    void *workspace;
};

struct GatedScanArgs {
    const void *x, *g;                        // [B, T, D], dtype dt (x may be null in a backward without input gate)
    const void *h, *dout;                     // backward only: the forward's output and its gradient
    const float *init_state, *dfinal;         // [N, D] fp32 or null
    const int32_t *cu;                        // [N + 1] or null
    void *out, *dx, *dg;                      // forward: out; backward: dx, dg; dtype dt
    float *final_state, *dinit;               // [N, D] fp32 or null
    int N, T, D, dt, input_gate;
};

struct LayerNormArgs {
    const void *x, *dout;                     // [rows, D], dtype dt
    const float *weight, *bias;               // [D] fp32 or null
    void *out, *dx;                           // [rows, D], dtype dt
    float *mean, *rstd;                       // [rows] fp32: written by the forward, read by the backward
    float *dweight, *dbias;                   // [D] fp32 or null
    int64_t rows;
    int D, dt;
    float eps;
    void *workspace;
};

struct RmsNormArgs {
    const void *x, *residual;                 // [rows, D], dtype dt; residual null or added, the sum going to residual_out
    const void *dout, *dresidual;             // backward: dtype dt, dresidual null or added to dx
    const float *weight;                      // [D] fp32 or null
    void *out, *residual_out, *dx;            // [rows, D], dtype dt; out e4m3 where scales is given
    float *scales;                            // [rows, ceil(D / 128)] fp32 or null
    float *rstd;                              // [rows] fp32: written by the forward (or null), read by the backward
    float *dweight;                           // [D] fp32 or null
    int64_t rows;
    int D, dt;
    float eps;
    void *workspace;
};

struct Fp8QuantArgs {
    const void *x;                            // [rows, D], dtype dt
    unsigned char *q;                         // [rows, D] e4m3
    float *scales;                            // [ceil(rows / block_rows), ceil(D / 128)]
    int64_t rows;
    int D, dt, block_rows;                    // 1 or 128
};

struct Fp8LinearArgs {
    const unsigned char *x, *w;               // [M, K], [N, K] e4m3
    const float *xs, *ws;                     // [M, ceil(K / 128)], [ceil(N / 128), ceil(K / 128)]
    void *out;                                // [M, N] bf16
    int M, N, K;
    void *workspace;
};

// What the log probabilities' forward call writes in place of loss and lse.
struct LogProbs {
    float *logp, *entropy, *lse;              // [N] fp32; lse may be null
    int32_t *top_ids;                         // [N, top_k]
    float *top_logps;                         // [N, top_k] fp32
    int top_k;
};

struct LinearCeArgs {
    const void *h, *w;                        // [N, D], [V, D], dtype dt
    const int32_t *targets;                   // [N]
    const float *lse_in, *dloss;              // backward only: [N] fp32
    float *loss, *lse;                        // forward only: [N] fp32
    void *dh, *dw;                            // backward only: [N, D], [V, D], dtype dt
    int N, D, V, dt;
    void *workspace;
};

// The log probabilities' backward call, beside dlogp in dloss: dloss counts with the sign -1, and a gradient of the entropy
// (else null) comes with the entropy, [N] fp32.
struct LogProbsGrad {
    const float *dentropy = nullptr, *entropy = nullptr;
    float sign = 1.f;
};

cudaError_t launch_gated_scan_fwd(const GatedScanArgs &a, cudaStream_t st);
cudaError_t launch_gated_scan_bwd(const GatedScanArgs &a, cudaStream_t st);
cudaError_t launch_gated_scan_step(float *state, const void *x, const void *g, void *out, int64_t n, int dt,
                                   int input_gate, cudaStream_t st);
cudaError_t launch_layer_norm_fwd(const LayerNormArgs &a, cudaStream_t st);
cudaError_t launch_layer_norm_bwd(const LayerNormArgs &a, cudaStream_t st);
size_t layer_norm_bwd_workspace_bytes(int64_t rows, int D, int dt);
cudaError_t launch_rms_norm_fwd(const RmsNormArgs &a, cudaStream_t st);
cudaError_t launch_rms_norm_bwd(const RmsNormArgs &a, cudaStream_t st);
size_t rms_norm_bwd_workspace_bytes(int D);
cudaError_t launch_fp8_quantize(const Fp8QuantArgs &a, cudaStream_t st);
cudaError_t launch_fp8_linear(const Fp8LinearArgs &a, cudaStream_t st);
// K a multiple of 16, tensors on 16-byte boundaries
bool fp8_linear_tc_supported(const Fp8LinearArgs &a);
// stall_ns: the self-test's; the first tile's data never comes, and waits give up after it
cudaError_t launch_fp8_linear_tc(const Fp8LinearArgs &a, cudaStream_t st, uint64_t stall_ns = 0);
size_t fp8_linear_workspace_bytes(int M, int N, int K);
// out, grad: the log probabilities' calls
cudaError_t launch_linear_ce_fwd(const LinearCeArgs &a, cudaStream_t st, const LogProbs *out = nullptr);
cudaError_t launch_linear_ce_bwd(const LinearCeArgs &a, cudaStream_t st, LogProbsGrad grad = LogProbsGrad());
// bf16 with D a multiple of 8 (rows that TMA can address) up to 2^24: the tensor cores
bool linear_ce_tc_supported(int dt, int D);
size_t linear_ce_tc_workspace_bytes(int N, int D, int V, bool backward, int top = -1);   // top: of log probabilities
// The self-test's: in this kernel (0 the logits, 1 E, 2 the gradients, 3 the log probabilities' logits) the first CTA pair's loads never come, and waits give
// up after limit_ns.
struct CeStall {
    int step = -1;
    uint64_t limit_ns = 0;
};
cudaError_t launch_linear_ce_tc_fwd(const LinearCeArgs &a, cudaStream_t st, const LogProbs *out = nullptr,
                                    CeStall stall = CeStall());
cudaError_t launch_linear_ce_tc_bwd(const LinearCeArgs &a, cudaStream_t st, LogProbsGrad grad = LogProbsGrad(),
                                    CeStall stall = CeStall());
size_t linear_ce_workspace_bytes(int N, int D, int V, int dt, bool backward, int top = -1);

cudaError_t launch_chunk_simt(const ChunkArgs &a, cudaStream_t st);
cudaError_t launch_chunk_bwd(const BwdArgs &a, cudaStream_t st);
size_t chunk_bwd_workspace_bytes(int64_t slots, int H, int dk, int dv);
cudaError_t launch_prologue(const PrologueArgs &a, cudaStream_t st);
bool chunk_tc_supported(int dt, int dk, int dv, int64_t tokens);
size_t chunk_tc_workspace_bytes(int64_t slots, int H, bool fused = false);
cudaError_t launch_chunk_tc(const ChunkArgs &a, cudaStream_t st);
cudaError_t launch_decode(const DecodeArgs &a, cudaStream_t st);
// one CTA whose bounded wait on a never-completed mbarrier phase gives up after limit_ns
cudaError_t launch_wait_selftest(unsigned *err, uint64_t limit_ns, cudaStream_t st);

}  // namespace gdn
