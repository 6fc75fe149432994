// C ABI of the decay attention, the layer norm and the 8-bit activations (see include/kda.h): argument
// checks, status codes, dispatch by type.  Nothing is launched before every check has passed.
#include <stdint.h>

#include "../../include/kda.h"
#include "kda_launch.h"

namespace kda {
namespace {

bool valid_dim(int d) { return d == 8 || d == 16 || d == 32 || d == 64 || d == 128; }
bool valid_dtype(int t) { return t == KDA_F32 || t == KDA_BF16; }
size_t esize(int dtype) { return dtype == KDA_BF16 ? 2 : 4; }

struct Buf {
  const void* p;
  size_t n;
};
bool overlap(const Buf& a, const Buf& b) {
  if (!a.p || !b.p || a.n == 0 || b.n == 0) return false;
  const uintptr_t x = (uintptr_t)a.p, y = (uintptr_t)b.p;
  return x < y + b.n && y < x + a.n;
}
// Every output against every input and every other output.
template <int NI, int NO> bool any_overlap(const Buf (&ins)[NI], const Buf (&outs)[NO]) {
  for (int i = 0; i < NO; ++i) {
    for (int j = 0; j < NI; ++j)
      if (overlap(outs[i], ins[j])) return true;
    for (int j = 0; j < i; ++j)
      if (overlap(outs[i], outs[j])) return true;
  }
  return false;
}
bool aligned(const void* p, size_t n) { return ((uintptr_t)p & (n - 1)) == 0; }

// (2^20 heads, so that no launch passes 2^32 threads)
bool attn_sizes(int B, int H, int T, int K, int V, int dtype) {
  return B >= 1 && H >= 1 && T >= 0 && valid_dim(K) && valid_dim(V) && (long long)B * H <= (1 << 20) &&
         ((size_t)T + 64) * (size_t)(K > V ? K : V) * esize(dtype) <= 0x7fffffffu;
}
size_t attn_states(int B, int H, int T, int K, int V, int dtype, bool bwd) {
  if (!valid_dtype(dtype) || !attn_sizes(B, H, T, K, V, dtype)) return 0;
  const DecayPlan p = decay_plan(B, H, T, K, V, dtype == KDA_BF16, bwd);
  return decay_states_bytes(B, H, K, V, p) * (bwd && p.nseg > 1 ? 2 : 1);
}
bool norm_sizes(int B, int H, int T, int D) {
  return B >= 1 && H >= 1 && T >= 0 && D >= 1 && D <= (1 << 24) && (long long)B * H <= (1 << 20) && (long long)H * D <= (1 << 28) &&
         (long long)B * H * T < 0x7fffffffLL;
}
int ckpt_group(int D) { return D < 32 ? D : 32; }

}  // namespace
}  // namespace kda

using namespace kda;

extern "C" {

size_t kda_decay_attn_workspace_bytes(int B, int H, int T, int K, int V, int dtype) {
  return attn_states(B, H, T, K, V, dtype, false);
}

int kda_decay_attn_fwd(const void* q, const void* k, const void* v, const float* log_decay, const int* lengths,
                       const float* state_in, float scale, void* o, float* state_out, void* workspace,
                       size_t workspace_bytes, int B, int H, int T, int K, int V, int dtype, void* stream) {
  if (!log_decay || (T != 0 && (!q || !k || !v || !o))) return reject(KDA_ERR_NULL);
  if (!valid_dtype(dtype)) return reject(KDA_ERR_DTYPE);
  if (!attn_sizes(B, H, T, K, V, dtype)) return reject(KDA_ERR_SHAPE);
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(o, 16)) return reject(KDA_ERR_ALIGN);
  const size_t need = attn_states(B, H, T, K, V, dtype, false);
  if (need && (!workspace || workspace_bytes < need)) return reject(KDA_ERR_WORKSPACE);
  if (need && !aligned(workspace, 256)) return reject(KDA_ERR_ALIGN);
  const size_t es = esize(dtype), bh = (size_t)B * H, ns = bh * K * V * 4;
  const Buf ins[] = {{q, bh * T * K * es}, {k, bh * T * K * es}, {v, bh * T * V * es}, {log_decay, (size_t)H * 4},
                     {lengths, (size_t)B * 4}, {state_in == state_out ? nullptr : state_in, ns}};
  const Buf outs[] = {{o, bh * T * V * es}, {state_out, ns}, {need ? workspace : nullptr, need}};
  if (any_overlap(ins, outs)) return reject(KDA_ERR_ALIAS);
  hipStream_t s = (hipStream_t)stream;
  const hipError_t e = dtype == KDA_BF16
                           ? launch_decay_fwd<bf16_t>(q, k, v, log_decay, lengths, state_in, scale, o, state_out,
                                                      workspace, B, H, T, K, V, s)
                           : launch_decay_fwd<float>(q, k, v, log_decay, lengths, state_in, scale, o, state_out,
                                                     workspace, B, H, T, K, V, s);
  if (e != hipSuccess) return reject(KDA_ERR_HIP);
  count_call(KDA_COUNTER_CHUNK_FWD);
  return KDA_OK;
}

int kda_decay_attn_step(const void* q, const void* k, const void* v, const float* log_decay, float* state,
                        float scale, void* o, int B, int H, int K, int V, int dtype, void* stream) {
  if (!q || !k || !v || !log_decay || !state || !o) return reject(KDA_ERR_NULL);
  if (!valid_dtype(dtype)) return reject(KDA_ERR_DTYPE);
  if (!attn_sizes(B, H, 1, K, V, dtype)) return reject(KDA_ERR_SHAPE);
  const size_t es = esize(dtype), bh = (size_t)B * H, ns = bh * K * V * 4;
  if (!aligned(state, 16) || !aligned(v, 16) || !aligned(q, es) || !aligned(k, es) || !aligned(o, es))
    return reject(KDA_ERR_ALIGN);
  const Buf ins[] = {{q, bh * K * es}, {k, bh * K * es}, {v, bh * V * es}, {log_decay, (size_t)H * 4}};
  const Buf outs[] = {{o, bh * V * es}, {state, ns}};
  if (any_overlap(ins, outs)) return reject(KDA_ERR_ALIAS);
  hipStream_t s = (hipStream_t)stream;
  const hipError_t e = dtype == KDA_BF16
                           ? launch_decay_step<bf16_t>(q, k, v, log_decay, state, scale, o, B, H, K, V, s)
                           : launch_decay_step<float>(q, k, v, log_decay, state, scale, o, B, H, K, V, s);
  if (e != hipSuccess) return reject(KDA_ERR_HIP);
  count_call(KDA_COUNTER_RECURRENT_STEP);
  return KDA_OK;
}

size_t kda_decay_attn_bwd_workspace_bytes(int B, int H, int T, int K, int V, int dtype) {
  return attn_states(B, H, T, K, V, dtype, true);
}

int kda_decay_attn_bwd(const void* q, const void* k, const void* v, const unsigned char* q_scales,
                       const unsigned char* k_scales, const unsigned char* v_scales, const float* log_decay,
                       const int* lengths, const float* state_in, float scale, const void* d_o,
                       const float* d_state_out, void* dq, void* dk, void* dv, float* dstate_in, void* workspace,
                       size_t workspace_bytes, int B, int H, int T, int K, int V, int dtype, void* stream) {
  if (!log_decay || !dstate_in || (T != 0 && (!q || !k || !v || !d_o || !dq || !dk || !dv)))
    return reject(KDA_ERR_NULL);
  if (T != 0 && ((q_scales != nullptr) != (k_scales != nullptr) || (q_scales != nullptr) != (v_scales != nullptr)))
    return reject(KDA_ERR_NULL);
  if (!valid_dtype(dtype)) return reject(KDA_ERR_DTYPE);
  if (!attn_sizes(B, H, T, K, V, dtype)) return reject(KDA_ERR_SHAPE);
  if (!aligned(q, q_scales ? 8 : 16) || !aligned(k, k_scales ? 8 : 16) || !aligned(v, v_scales ? 8 : 16) ||
      !aligned(d_o, 16) || !aligned(dq, 16) || !aligned(dk, 16) || !aligned(dv, 16))
    return reject(KDA_ERR_ALIGN);
  const size_t need = attn_states(B, H, T, K, V, dtype, true);
  if (need && (!workspace || workspace_bytes < need)) return reject(KDA_ERR_WORKSPACE);
  if (need && !aligned(workspace, 256)) return reject(KDA_ERR_ALIGN);
  const size_t es = esize(dtype), bh = (size_t)B * H, ns = bh * K * V * 4;
  const size_t nk = bh * T * K, nv = bh * T * V;
  const size_t gk = bh * T * (K / ckpt_group(K)), gv = bh * T * (V / ckpt_group(V));
  const Buf ins[] = {{q, nk * (q_scales ? 1 : es)}, {k, nk * (k_scales ? 1 : es)}, {v, nv * (v_scales ? 1 : es)},
                     {q_scales, gk}, {k_scales, gk}, {v_scales, gv}, {log_decay, (size_t)H * 4},
                     {lengths, (size_t)B * 4}, {state_in, ns}, {d_o, nv * es}, {d_state_out, ns}};
  const Buf outs[] = {{dq, nk * es}, {dk, nk * es}, {dv, nv * es}, {dstate_in, ns}, {need ? workspace : nullptr, need}};
  if (any_overlap(ins, outs)) return reject(KDA_ERR_ALIAS);
  hipStream_t s = (hipStream_t)stream;
  const hipError_t e =
      dtype == KDA_BF16
          ? launch_decay_bwd<bf16_t>(q, k, v, q_scales, k_scales, v_scales, log_decay, lengths, state_in, scale, d_o,
                                     d_state_out, dq, dk, dv, dstate_in, workspace, B, H, T, K, V, s)
          : launch_decay_bwd<float>(q, k, v, q_scales, k_scales, v_scales, log_decay, lengths, state_in, scale, d_o,
                                    d_state_out, dq, dk, dv, dstate_in, workspace, B, H, T, K, V, s);
  if (e != hipSuccess) return reject(KDA_ERR_HIP);
  count_call(KDA_COUNTER_CHUNK_BWD);
  return KDA_OK;
}

int kda_layer_norm_fwd(const void* x, const float* weight, const float* bias, float eps, void* y, float* mean,
                       float* rstd, int B, int H, int T, int D, int dtype, void* stream) {
  if (T != 0 && (!x || !y)) return reject(KDA_ERR_NULL);
  if (!valid_dtype(dtype)) return reject(KDA_ERR_DTYPE);
  if (!norm_sizes(B, H, T, D) || !(eps >= 0.0f && eps <= 3.0e38f)) return reject(KDA_ERR_SHAPE);
  const size_t es = esize(dtype), rows = (size_t)B * H * T, np = (size_t)H * D * 4;
  if (!aligned(x, es) || !aligned(y, es)) return reject(KDA_ERR_ALIGN);
  const Buf ins[] = {{x, rows * D * es}, {weight, np}, {bias, np}};
  const Buf outs[] = {{y, rows * D * es}, {mean, rows * 4}, {rstd, rows * 4}};
  if (any_overlap(ins, outs)) return reject(KDA_ERR_ALIAS);
  hipStream_t s = (hipStream_t)stream;
  const hipError_t e = dtype == KDA_BF16 ? launch_norm_fwd<bf16_t>(x, weight, bias, eps, y, mean, rstd, B, H, T, D, s)
                                         : launch_norm_fwd<float>(x, weight, bias, eps, y, mean, rstd, B, H, T, D, s);
  return e == hipSuccess ? KDA_OK : reject(KDA_ERR_HIP);
}

size_t kda_layer_norm_bwd_workspace_bytes(int B, int H, int T, int D, int dtype) {
  if (!valid_dtype(dtype) || !norm_sizes(B, H, T, D)) return 0;
  return norm_bwd_workspace_bytes(B, H, T, D, dtype == KDA_BF16);
}

int kda_layer_norm_bwd(const void* x, const unsigned char* x_scales, const float* weight, const float* mean,
                       const float* rstd, const void* dy, void* dx, float* dweight, float* dbias, void* workspace,
                       size_t workspace_bytes, int B, int H, int T, int D, int dtype, void* stream) {
  if (T != 0 && (!x || !mean || !rstd || !dy || !dx)) return reject(KDA_ERR_NULL);
  if (!valid_dtype(dtype)) return reject(KDA_ERR_DTYPE);
  if (!norm_sizes(B, H, T, D) || (x_scales && D > 32 && D % 32)) return reject(KDA_ERR_SHAPE);
  const size_t es = esize(dtype), rows = (size_t)B * H * T, np = (size_t)H * D * 4;
  if (!aligned(x, x_scales ? 1 : es) || !aligned(dy, es) || !aligned(dx, es)) return reject(KDA_ERR_ALIGN);
  const size_t need = (dweight || dbias) ? kda_layer_norm_bwd_workspace_bytes(B, H, T, D, dtype) : 0;
  if (need && (!workspace || workspace_bytes < need)) return reject(KDA_ERR_WORKSPACE);
  if (need && !aligned(workspace, 16)) return reject(KDA_ERR_ALIGN);
  const Buf ins[] = {{x, rows * D * (x_scales ? 1 : es)}, {x_scales, rows * (D / ckpt_group(D))}, {weight, np},
                     {mean, rows * 4}, {rstd, rows * 4}, {dx == dy ? nullptr : dy, rows * D * es}};
  const Buf outs[] = {{dx, rows * D * es}, {dweight, np}, {dbias, np}, {need ? workspace : nullptr, need}};
  if (any_overlap(ins, outs)) return reject(KDA_ERR_ALIAS);
  hipStream_t s = (hipStream_t)stream;
  const hipError_t e = dtype == KDA_BF16 ? launch_norm_bwd<bf16_t>(x, x_scales, weight, mean, rstd, dy, dx, dweight,
                                                                   dbias, workspace, B, H, T, D, s)
                                         : launch_norm_bwd<float>(x, x_scales, weight, mean, rstd, dy, dx, dweight,
                                                                  dbias, workspace, B, H, T, D, s);
  return e == hipSuccess ? KDA_OK : reject(KDA_ERR_HIP);
}

static int ckpt_checks(const void* x, const void* codes, const void* scales, long long rows, int D, int dtype) {
  if (rows != 0 && (!x || !codes || !scales)) return KDA_ERR_NULL;
  if (!valid_dtype(dtype)) return KDA_ERR_DTYPE;
  if (rows < 0 || D < 1 || (D > 32 && D % 32) || D > (1 << 24) || rows > (1LL << 50) / D) return KDA_ERR_SHAPE;
  if (!aligned(x, esize(dtype))) return KDA_ERR_ALIGN;
  const size_t n = (size_t)rows * D, g = (size_t)rows * (D / ckpt_group(D));
  if (overlap({x, n * esize(dtype)}, {codes, n}) || overlap({x, n * esize(dtype)}, {scales, g}) ||
      overlap({codes, n}, {scales, g}))
    return KDA_ERR_ALIAS;
  return KDA_OK;
}

int kda_ckpt_pack(const void* x, unsigned char* codes, unsigned char* scales, long long rows, int D, int dtype,
                  void* stream) {
  const int st = ckpt_checks(x, codes, scales, rows, D, dtype);
  if (st != KDA_OK) return reject(st);
  hipStream_t s = (hipStream_t)stream;
  const hipError_t e = dtype == KDA_BF16 ? launch_ckpt_pack<bf16_t>(x, codes, scales, rows, D, s)
                                         : launch_ckpt_pack<float>(x, codes, scales, rows, D, s);
  return e == hipSuccess ? KDA_OK : reject(KDA_ERR_HIP);
}

int kda_ckpt_unpack(const unsigned char* codes, const unsigned char* scales, void* x, long long rows, int D,
                    int dtype, void* stream) {
  const int st = ckpt_checks(x, codes, scales, rows, D, dtype);
  if (st != KDA_OK) return reject(st);
  hipStream_t s = (hipStream_t)stream;
  const hipError_t e = dtype == KDA_BF16 ? launch_ckpt_unpack<bf16_t>(codes, scales, x, rows, D, s)
                                         : launch_ckpt_unpack<float>(codes, scales, x, rows, D, s);
  return e == hipSuccess ? KDA_OK : reject(KDA_ERR_HIP);
}

}  // extern "C"
