// Host-side launchers of the KDA kernels (definitions in the .hip files).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>

#include "kda_common.h"

namespace kda {

template <typename Tin>
hipError_t launch_gate(const void* z, const float* A_log, const float* dt_bias, float* g, float* alpha, int B, int H,
                       int T, int K, hipStream_t s);

// Gate adjoint: dz (nullable), dA_log and d_dt_bias (nullable) for a cotangent dg.
size_t gate_bwd_workspace_bytes(int B, int H, int T, int K);
// Device address of the current device's built-in gate-adjoint scratch
// (KDA_GATE_BWD_SCRATCH_BYTES), looked up once per device.
hipError_t gate_bwd_scratch(void** ptr);
template <typename Tin>
hipError_t launch_gate_bwd(const void* z, const float* A_log, const float* dt_bias, const float* dg, float* dz,
                           float* dA_log, float* d_dt_bias, void* workspace, int B, int H, int T, int K,
                           hipStream_t s);

template <typename Tin>
hipError_t launch_step(const void* q, const void* k, const void* v, const void* z, const float* A_log,
                       const float* dt_bias, const void* beta, float* state, float scale, void* o, int B, int H,
                       int K, int V, int zc, hipStream_t s);

// Gate layout of the forward and step launchers: zc = 1, z is (B,H,T,K) and dt_bias (H,K);
// zc = 0, the scalar-decay case, z is (B,H,T) and dt_bias (H).

// Chunked forward: instance chosen by (padded key dim KD, value tile VT, chunk C).
// ckpt (nullable) receives the state at every chunk start: (B,H,ceil(T/C),K,V) fp32.
template <typename Tin, int KD>
hipError_t launch_chunk_fwd_kd(int VT, int C, const void* q, const void* k, const void* v, const void* z,
                               const float* A_log, const float* dt_bias, const void* beta, const float* state_in,
                               float scale, void* o, float* state_out, float* ckpt, int B, int H, int T, int K, int V,
                               int zc, hipStream_t s);

// Pipelined bf16 forward (16 waves, internal blocks of C <= 32 tokens).
template <int KD>
hipError_t launch_chunk_fwd_pc_kd(int VT, int C, const void* q, const void* k, const void* v, const void* z,
                                  const float* A_log, const float* dt_bias, const void* beta, const float* state_in,
                                  float scale, void* o, float* state_out, int B, int H, int T, int K, int V, int zc,
                                  hipStream_t s);

// Paired bf16 forward for V = 128 (two workgroups per head share the gate and WY work
// through a ring in `work`, px_workspace_bytes() of it; see kda_chunk_fwd_px.h).
template <int KD>
hipError_t launch_chunk_fwd_px_kd(const void* q, const void* k, const void* v, const void* z, const float* A_log,
                                  const float* dt_bias, const void* beta, const float* state_in, float scale, void* o,
                                  float* state_out, int B, int H, int T, int K, int zc, void* work,
                                  unsigned long long spin_ticks, hipStream_t s);
size_t px_workspace_bytes(int KD, int nheads);

// The bf16 forward with the output RMSNorm fused into its output stage (o holds
// y = o / sqrt(mean_v o^2 + eps) * norm_w[h]); when V > 64 the two value tiles of a head
// exchange per-token sums of squares through `work` (norm_workspace_bytes() of it).
template <int KD>
hipError_t launch_chunk_fwd_norm_kd(const void* q, const void* k, const void* v, const void* z, const float* A_log,
                                    const float* dt_bias, const void* beta, const float* state_in, float scale,
                                    const float* norm_w, float eps, void* o, float* state_out, int B, int H, int T,
                                    int K, int V, void* work, unsigned long long spin_ticks, hipStream_t s);
size_t norm_workspace_bytes(int B, int H, int T, int V);

// Forward tiling actually used for (dtype, K, V, chunk): padded key dim, value tile
// and the chunk the kernel blocks by.  Returns false when no instance exists.
struct FwdPlan {
  int KD, VT, C;
};
bool fwd_plan(bool bf16, int K, int V, int chunk, FwdPlan* plan);

// Chunked adjoint on MFMA (fp32 activations), see kda_bwd_chunk.hip.
size_t chunk_bwd_mfma_workspace_bytes(int B, int H, int T, int K, int V);
hipError_t launch_chunk_bwd_mfma(const float* q, const float* k, const float* v, const float* z, const float* A_log,
                                 const float* dt_bias, const float* beta, const float* state_in, float scale,
                                 const float* d_o, const float* d_state_out, float* dq, float* dk, float* dv,
                                 float* dg, float* dbeta, float* dstate_in, void* workspace, int B, int H, int T,
                                 int K, int V, hipStream_t s);

// Linear attention with a constant decay per head (kda_decay_attn.hip).  The tokens are walked in nseg
// segments of seglen tokens; nseg > 1 needs the segments' states in a workspace (two of them backward).
// A backward pass with nseg = 1 may still cut the walk of dv, into vseg segments of vlen tokens (vseg > 1).
struct DecayPlan {
  int nseg, seglen, vseg, vlen;
};
DecayPlan decay_plan(int B, int H, int T, int K, int V, bool bf16, bool bwd);
size_t decay_states_bytes(int B, int H, int K, int V, const DecayPlan& p);   // of S, and of dL/dS backward
template <typename T>
hipError_t launch_decay_fwd(const void* q, const void* k, const void* v, const float* log_decay, const int* lengths,
                            const float* state_in, float scale, void* o, float* state_out, void* workspace, int B,
                            int H, int T_, int K, int V, hipStream_t s);
template <typename T>
hipError_t launch_decay_bwd(const void* q, const void* k, const void* v, const uint8_t* q_sc, const uint8_t* k_sc,
                            const uint8_t* v_sc, const float* log_decay, const int* lengths, const float* state_in,
                            float scale, const void* d_o, const float* d_state_out, void* dq, void* dk, void* dv,
                            float* dstate_in, void* workspace, int B, int H, int T_, int K, int V, hipStream_t s);
template <typename T>
hipError_t launch_decay_step(const void* q, const void* k, const void* v, const float* log_decay, float* state,
                             float scale, void* o, int B, int H, int K, int V, hipStream_t s);

// Layer norm (kda_layer_norm.hip); x_scales non-null: x holds 8-bit codes.
template <typename T>
hipError_t launch_norm_fwd(const void* x, const float* w, const float* b, float eps, void* y, float* mean, float* rstd,
                           int B, int H, int T_, int D, hipStream_t s);
size_t norm_bwd_workspace_bytes(int B, int H, int T, int D, bool bf16);
template <typename T>
hipError_t launch_norm_bwd(const void* x, const uint8_t* x_scales, const float* w, const float* mean,
                           const float* rstd, const void* dy, void* dx, float* dw, float* db, void* workspace, int B,
                           int H, int T_, int D, hipStream_t s);

// 8-bit activations (kda_ckpt.hip).
template <typename T>
hipError_t launch_ckpt_pack(const void* x, uint8_t* codes, uint8_t* scales, long long rows, int D, hipStream_t s);
template <typename T>
hipError_t launch_ckpt_unpack(const uint8_t* codes, const uint8_t* scales, void* x, long long rows, int D,
                              hipStream_t s);

// Short causal convolution (kda_short_conv.hip): x (B, T, C = H D) at strides xb, xt; y, dy (B, H, T, D).
template <typename T>
hipError_t launch_conv_fwd(const void* x, long long xb, long long xt, const float* w, const float* bias,
                           const int* lengths, const void* state_in, int silu, void* y, void* state_out, int B, int H,
                           int T_, int D, int W, hipStream_t s);
template <typename T>
hipError_t launch_conv_step(const void* x, long long xb, const float* w, const float* bias, int silu, void* state,
                            void* y, int B, int C, int W, hipStream_t s);
size_t conv_bwd_workspace_bytes(int B, int H, int T, int D, int W, bool bf16);
template <typename T>
hipError_t launch_conv_bwd(const void* x, long long xb, long long xt, const float* w, const float* bias,
                           const int* lengths, const void* state_in, int silu, const void* dy, const float* d_state,
                           void* dx, long long dxb, long long dxt, float* dw, float* db, float* d_state_in,
                           void* workspace, int B, int H, int T_, int D, int W, hipStream_t s);

// Norm of queries and keys with their rotation (kda_qk_rope.hip): [0] the queries, [1] the keys (H = 0: none).
struct QkSideDesc {
  const void* x;
  long long xb, xt, xh;        // strides of the batch, the token and the head, in elements
  const float* w;              // (Hw, D) or null; per_head: Hw = H, not one row for all heads
  int H, per_head;
  void* y;                     // forward: out; backward: the cotangent
  void* dx;
  long long db, dt, dh;
};
template <typename T>
hipError_t launch_qk_fwd(const QkSideDesc* d, const double* freqs, const int* positions, int norm, float eps,
                         float rope_scale, int interleaved, int B, int T_, int D, int R, hipStream_t s);
size_t qk_bwd_workspace_bytes(int B, int T, int Hq, int Hk, int D, int q_per_head, int k_per_head);
template <typename T>
hipError_t launch_qk_bwd(const QkSideDesc* d, const double* freqs, const int* positions, int norm, float eps,
                         float rope_scale, int interleaved, float* dwq, float* dwk, void* workspace, int B, int T_,
                         int D, int R, hipStream_t s);

// Gated linear recurrence (kda_gated_scan.hip); i null: no input gate; ckpt null: not kept.
size_t scan_workspace_bytes(int B, int H, int T, int D, bool bf16);
size_t scan_bwd_workspace_bytes(int B, int H, int T, int D, bool bf16);
template <typename T>
hipError_t launch_scan_fwd(const void* x, const void* z, const float* A_log, const float* dt_bias, const void* i,
                           const int* lengths, const float* state_in, int normalize, void* y, float* state_out,
                           float* ckpt, void* workspace, int B, int H, int T_, int D, hipStream_t s);
template <typename T>
hipError_t launch_scan_step(const void* x, const void* z, const float* A_log, const float* dt_bias, const void* i,
                            int normalize, float* state, void* y, int B, int H, int D, hipStream_t s);
template <typename T>
hipError_t launch_scan_bwd(const void* x, const void* z, const float* A_log, const float* dt_bias, const void* i,
                           const int* lengths, int normalize, const float* ckpt, const void* dy, const float* d_state,
                           void* dx, void* dz, void* di, float* dA_log, float* d_dt_bias, float* d_state_in,
                           void* workspace, int B, int H, int T_, int D, hipStream_t s);

// Counters of kda_api.hip: a rejected call (returns its status), an accepted one.
int reject(int status);
void count_call(int counter);

}  // namespace kda
