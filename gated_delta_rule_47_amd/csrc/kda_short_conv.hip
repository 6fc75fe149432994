// Short causal depthwise convolution of a projection with its activation, its single-token form and its adjoint.
//
//   pre_t = bias + sum_j w_j x_{t - W + 1 + j},  y_t = act(pre_t)              (j = 0 .. W - 1 per channel)
//   dpre_t = dy_t act'(pre_t),  dx_t = sum_j w_j dpre_{t + W - 1 - j},  dw_j = sum_t dpre_t x_{t - W + 1 + j}
//
// Memory is what bounds all three: x (and dy) read once, y (or dx) written once.  A lane holds a few neighbouring
// channels and walks a run of tokens with the last W - 1 inputs in registers, so a row is read once per run but
// for W - 1 rows in front (backward: and behind) of it.  64 lanes take 64 neighbouring groups of channels
// (contiguous rows of a wave), the workgroup's waves neighbouring runs.  y is written head by head.
// Measured: forward, 2 x 16384 tokens of 4096 channels, W = 4, bf16, 109 us (4.9 TB/s), half as many in fp32 106; one token of
// 192 x 12288, 10 us (3.7 TB/s, 4 of them the kernel's start); adjoint, 2 x 8192 x 4096, bf16, 88 us (4.6 TB/s), a padded
// batch of 8 x 4096 x 512, where few waves have work, 26 and 4 for the sums.
#include "kda_launch.h"
#include "kda_vec.h"

namespace kda {
namespace {

constexpr int kConvThreads = 256, kConvStepBatch = 2;

__device__ __forceinline__ float sigmoid_f(float x) { return fast_rcp(1.0f + fast_exp2(-kLog2e * x)); }

struct ConvArgs {
  const void* x;
  long long xb, xt;            // strides of the batch and of the token, in elements
  const float *w, *bias;
  const int* lengths;
  const void* state_in;        // (B, W - 1, C)
  void* y;
  void* state_out;
  const void* dy;              // backward
  const float* d_state;
  void* dx;
  long long db, dt;
  float *parts, *d_state_in;
  int B, H, T, D, C, silu;
  int lanes_log2, run, blocks_t;   // lanes per run, tokens per run, workgroups along a sequence
};

__device__ __forceinline__ int length_of(const ConvArgs& a, int b) {
  return a.lengths ? min(max(a.lengths[b], 0), a.T) : a.T;
}

// Where a workgroup's lane stands: its channels, its sequence, its run's first token.
struct ConvPlace {
  int c, b, t0, tb;
  bool on;
};
template <int E> __device__ __forceinline__ ConvPlace conv_place(const ConvArgs& a) {
  const int lanes = 1 << a.lanes_log2, runs = kConvThreads >> a.lanes_log2;
  const int lane = threadIdx.x & (lanes - 1), r = threadIdx.x >> a.lanes_log2;
  const int cblocks = (a.C / E + lanes - 1) >> a.lanes_log2;
  unsigned id = blockIdx.x;
  ConvPlace p;
  p.c = ((id % cblocks << a.lanes_log2) + lane) * E;
  id /= cblocks;
  p.tb = id % a.blocks_t;
  p.b = id / a.blocks_t;
  p.t0 = (p.tb * runs + r) * a.run;      // < T + runs * run, within an int (T <= 2^28)
  p.on = p.c < a.C;
  return p;
}

// Row t >= -(W - 1) of a sequence's inputs: the tokens behind the kept inputs before them.
template <typename T, int W, int E>
__device__ __forceinline__ void conv_row(const ConvArgs& a, int b, int c, long long t, Elems<T, E>& r) {
  if (t >= 0) r.load((const T*)a.x + b * a.xb + t * a.xt + c);
  else if (a.state_in) r.load((const T*)a.state_in + ((size_t)b * (W - 1) + (W - 1 + t)) * a.C + c);
  else r.zero();
}

template <int W, int E> __device__ __forceinline__ void conv_weights(const ConvArgs& a, int c, float (&w)[W][E], float (&bias)[E]) {
  float f[W * E];
  load_f32<W * E>(a.w + (size_t)c * W, f);
#pragma unroll
  for (int e = 0; e < E; ++e)
#pragma unroll
    for (int j = 0; j < W; ++j) w[j][e] = f[e * W + j];
  if (a.bias) load_f32<E>(a.bias + c, bias);
  else
#pragma unroll
    for (int e = 0; e < E; ++e) bias[e] = 0.f;
}

template <typename T, int W, int E> __global__ __launch_bounds__(kConvThreads) void conv_fwd_kernel(ConvArgs a) {
  const ConvPlace p = conv_place<E>(a);
  if (!p.on) return;
  const int n = length_of(a, p.b), t1 = min(p.t0 + a.run, n);
  if (p.t0 < t1) {
    float w[W][E], bias[E], win[W][E];
    conv_weights<W, E>(a, p.c, w, bias);
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
      Elems<T, E> r;
      conv_row<T, W, E>(a, p.b, p.c, p.t0 - (W - 1) + j, r);
#pragma unroll
      for (int e = 0; e < E; ++e) win[j][e] = r.at(e);
    }
    const T* x = (const T*)a.x + p.b * a.xb + p.t0 * a.xt + p.c;
    T* y = (T*)a.y + (((size_t)p.b * a.H + p.c / a.D) * a.T + p.t0) * a.D + p.c % a.D;
    constexpr int U = sizeof(T) == 2 ? 8 : 4;
    for (int t = p.t0; t < t1; t += U, x += U * a.xt, y += (size_t)U * a.D) {
      Elems<T, E> raw[U];
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (t + u < t1) raw[u].load(x + u * a.xt);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (t + u >= t1) break;
        float o[E];
#pragma unroll
        for (int e = 0; e < E; ++e) {
          win[W - 1][e] = raw[u].at(e);
          float s = bias[e];
#pragma unroll
          for (int j = 0; j < W; ++j) s = fmaf(w[j][e], win[j][e], s);
          o[e] = a.silu ? s * sigmoid_f(s) : s;
#pragma unroll
          for (int j = 0; j < W - 1; ++j) win[j][e] = win[j + 1][e];
        }
        Elems<T, E> out;
        out.set(o);
        out.store(y + (size_t)u * a.D);
      }
    }
  }
  // the run that holds the sequence's last token keeps the W - 1 inputs in front of its end
  if (a.state_out && p.t0 <= max(n - 1, 0) && max(n - 1, 0) < p.t0 + a.run)
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
      Elems<T, E> r;
      conv_row<T, W, E>(a, p.b, p.c, (long long)n - (W - 1) + j, r);
      r.store((T*)a.state_out + ((size_t)p.b * (W - 1) + j) * a.C + p.c);
    }
}

// One token: the state's rows move up by one.  A lane takes NB sequences of its channels, whose weights it reads once.
template <typename T, int W, int E> __global__ __launch_bounds__(kConvThreads) void conv_step_kernel(ConvArgs a) {
  constexpr int NB = kConvStepBatch;
  const unsigned id = blockIdx.x * kConvThreads + threadIdx.x, vecs = a.C / E;
  const unsigned b0 = id / vecs * NB;
  const int c = (int)(id % vecs) * E;
  if (b0 >= (unsigned)a.B) return;
  Elems<T, E> row[NB][W];
#pragma unroll
  for (int k = 0; k < NB; ++k) {
    if (b0 + k >= (unsigned)a.B) break;
    const T* state = (const T*)a.state_out + (size_t)(b0 + k) * (W - 1) * a.C + c;
    row[k][W - 1].load((const T*)a.x + (b0 + k) * a.xb + c);
#pragma unroll
    for (int j = 0; j < W - 1; ++j) row[k][j].load(state + (size_t)j * a.C);
  }
  float w[W][E], bias[E];
  conv_weights<W, E>(a, c, w, bias);
#pragma unroll
  for (int k = 0; k < NB; ++k) {
    if (b0 + k >= (unsigned)a.B) break;
    T* state = (T*)a.state_out + (size_t)(b0 + k) * (W - 1) * a.C + c;
    float o[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
      o[e] = bias[e];
#pragma unroll
      for (int j = 0; j < W; ++j) o[e] = fmaf(w[j][e], row[k][j].at(e), o[e]);
      if (a.silu) o[e] *= sigmoid_f(o[e]);
    }
    Elems<T, E> out;
    out.set(o);
    out.store((T*)a.y + (size_t)(b0 + k) * a.C + c);
#pragma unroll
    for (int j = 0; j < W - 1; ++j) row[k][j + 1].store(state + (size_t)j * a.C);
  }
}

// What a run of the adjoint holds in registers: weights, the last W - 1 inputs and cotangents, its sums.
template <int W, int E> struct ConvRun {
  float w[W][E], bias[E], win[W][E], dp[W][E], dw[W][E], db[E];
};

// One token: its cotangent dpre (0 behind the sequence), its share of the sums, and in o the gradient of the input W - 1
// tokens before it, which is complete with it.
template <bool SILU, bool FAST, int W, int E, typename RT>
__device__ __forceinline__ void conv_bwd_token(ConvRun<W, E>& c, const RT& rx, const RT& rd, bool inside, bool own, float (&o)[E]) {
#pragma unroll
  for (int e = 0; e < E; ++e) {
    c.win[W - 1][e] = rx.at(e);
    float d = rd.at(e);
    if constexpr (SILU) {
      float s = c.bias[e];
#pragma unroll
      for (int j = 0; j < W; ++j) s = fmaf(c.w[j][e], c.win[j][e], s);
      const float g = sigmoid_f(s);
      d *= fmaf(s, g * (1.f - g), g);
    }
    if (!FAST && !inside) d = 0.f;
    c.dp[W - 1][e] = d;
    if (FAST || (inside && own)) {
      c.db[e] += d;
#pragma unroll
      for (int j = 0; j < W; ++j) c.dw[j][e] = fmaf(d, c.win[j][e], c.dw[j][e]);
    }
    o[e] = 0.f;
#pragma unroll
    for (int k = 0; k < W; ++k) o[e] = fmaf(c.w[W - 1 - k][e], c.dp[k][e], o[e]);
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
      c.win[j][e] = c.win[j + 1][e];
      c.dp[j][e] = c.dp[j + 1][e];
    }
  }
}

// Tokens t0 .. t0 + run - 1 give their dx and their share of dw and db; dpre is computed for W - 1 tokens more.  The
// tokens in the middle of a run inside its sequence take a path without conditions.
template <typename T, int W, int E, bool SILU> __global__ __launch_bounds__(kConvThreads) void conv_bwd_kernel(ConvArgs a) {
  __shared__ float red[kConvThreads * (W + 1) * E];
  const ConvPlace p = conv_place<E>(a);
  ConvRun<W, E> c;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    c.db[e] = 0.f;
#pragma unroll
    for (int j = 0; j < W; ++j) c.dw[j][e] = 0.f;
  }
  const int n = p.on ? length_of(a, p.b) : 0, own = min(p.t0 + a.run, a.T);
  if (p.on && p.t0 > 0 && p.t0 >= n) {                 // a run behind its sequence
    Elems<T, E> zero;
    zero.zero();
    T* dx = (T*)a.dx + p.b * a.db + p.t0 * a.dt + p.c;
    for (int t = p.t0; t < own; ++t, dx += a.dt) zero.store(dx);
  } else if (p.on) {
    const int t1 = own + W - 1, in = min(n, t1);       // tokens whose inputs are read: t < in
    conv_weights<W, E>(a, p.c, c.w, c.bias);
    const T* x = (const T*)a.x + p.b * a.xb + p.t0 * a.xt + p.c;
    const T* dy = (const T*)a.dy + (((size_t)p.b * a.H + p.c / a.D) * a.T + p.t0) * a.D + p.c % a.D;
    T* dx = (T*)a.dx + p.b * a.db + ((long long)p.t0 - (W - 1)) * a.dt + p.c;
    constexpr int U = 4;
    // the next U tokens' rows are on their way while these are worked on
    Elems<T, E> nx[U], nd[U];
    const auto fetch = [&](int t) {
      if (t + U <= in) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
          nx[u].load(x + u * a.xt);
          nd[u].load(dy + (size_t)u * a.D);
        }
      } else {
#pragma unroll
        for (int u = 0; u < U; ++u) {
          nx[u].zero();
          nd[u].zero();
          if (t + u < in) {
            nx[u].load(x + u * a.xt);
            nd[u].load(dy + (size_t)u * a.D);
          }
        }
      }
      x += U * a.xt;
      dy += (size_t)U * a.D;
    };
    fetch(p.t0);
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
      Elems<T, E> r;
      r.zero();
      if (p.t0 - (W - 1) + j < n) conv_row<T, W, E>(a, p.b, p.c, p.t0 - (W - 1) + j, r);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        c.win[j][e] = r.at(e);
        c.dp[j][e] = 0.f;                // (of tokens whose inputs' gradients are another run's, or in front of the first)
      }
    }
    for (int t = p.t0; t < t1; t += U, dx += U * a.dt) {
      Elems<T, E> rx[U], rd[U];
#pragma unroll
      for (int u = 0; u < U; ++u) rx[u] = nx[u], rd[u] = nd[u];
      fetch(t + U);
      if (t >= p.t0 + W - 1 && t + U <= min(n, own)) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
          float o[E];
          conv_bwd_token<SILU, true>(c, rx[u], rd[u], true, true, o);
          Elems<T, E> out;
          out.set(o);
          out.store(dx + u * a.dt);
        }
        continue;
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int r = t + u - (W - 1);   // the row whose gradient is complete with this token
        if (t + u >= t1) break;
        float o[E];
        conv_bwd_token<SILU, false>(c, rx[u], rd[u], t + u < n, t + u < own, o);
        if (a.d_state && r < n && r >= n - (W - 1)) {
          float f[E];
          load_f32<E>(a.d_state + ((size_t)p.b * (W - 1) + (r - n + W - 1)) * a.C + p.c, f);
#pragma unroll
          for (int e = 0; e < E; ++e) o[e] += f[e];
        }
        if (r >= p.t0) {
          Elems<T, E> out;
          out.set(o);
          out.store(dx + u * a.dt);
        } else if (r < 0) {              // (the first run only)
          Elems<float, E> out;
          out.set(o);
          out.store(a.d_state_in + ((size_t)p.b * (W - 1) + (W - 1 + r)) * a.C + p.c);
        }
      }
    }
  }
  if (!a.parts) return;
  // the runs' sums of the workgroup, in ascending order
  float* mine = red + threadIdx.x;       // [value][thread]
#pragma unroll
  for (int e = 0; e < E; ++e) {
#pragma unroll
    for (int j = 0; j < W; ++j) mine[(j * E + e) * kConvThreads] = c.dw[j][e];
    mine[(W * E + e) * kConvThreads] = c.db[e];
  }
  __syncthreads();
  const int lanes = 1 << a.lanes_log2, runs = kConvThreads >> a.lanes_log2;
  float* out = a.parts + ((size_t)p.b * a.blocks_t + p.tb) * (W + 1) * a.C;
  const int c0 = p.c - (threadIdx.x & (lanes - 1)) * E;
  for (int i = threadIdx.x; i < lanes * E * (W + 1); i += kConvThreads) {
    const int j = i >> a.lanes_log2, l = i & (lanes - 1);      // value j = tap * E + e of lane l
    float s = 0.f;
    for (int r = 0; r < runs; ++r) s += red[j * kConvThreads + (r << a.lanes_log2) + l];
    const int c = c0 + l * E + j % E;
    if (c < a.C) out[(size_t)(j / E) * a.C + c] = s;
  }
}

template <int W> __global__ __launch_bounds__(kSumThreads) void conv_params_kernel(const float* parts, int n_parts, int C,
                                                                                   float* dw, float* db) {
  sum_parts(parts, (size_t)(W + 1) * C, n_parts, (W + 1) * C, [=](int i, float s) {
    const int j = i / C, c = i % C;
    if (j < W) {
      if (dw) dw[(size_t)c * W + j] = s;
    } else if (db) {
      db[c] = s;
    }
  });
}

template <typename T> constexpr int conv_e(bool bwd) { return bwd || sizeof(T) == 4 ? 4 : 8; }

// Lanes along the channels (all of them, up to a wave), tokens of a run: about 2^17 lanes over the chip (8 waves per
// CU, which a run of 128 tokens keeps in flight; 2^18 lanes: forward 124 for 109 us at 2 x 16384 x 4096, backward 95 for 93 at
// 2 x 8192 x 4096), a run of 8 to 128 tokens, longer where the grid would pass 2^23 workgroups.
void conv_plan(ConvArgs& a, int E) {
  const int vecs = a.C / E;
  a.lanes_log2 = 0;
  while (a.lanes_log2 < 6 && (1 << a.lanes_log2) < vecs) ++a.lanes_log2;
  const int lanes = 1 << a.lanes_log2, runs = kConvThreads / lanes;
  const long long cblocks = (vecs + lanes - 1) / lanes;
  long long run = 8;
  while (run < 128 && (long long)a.B * a.T / run * vecs > (1 << 17)) run *= 2;
  while (a.B * cblocks * ((a.T + run * runs - 1) / (run * runs)) > (1 << 23) && run * runs < a.T) run *= 2;
  a.run = (int)run;
  a.blocks_t = (int)((a.T + run * runs - 1) / (run * runs));
  if (a.blocks_t < 1) a.blocks_t = 1;    // an empty call still copies the state
}
unsigned conv_grid(const ConvArgs& a, int E) {
  const int lanes = 1 << a.lanes_log2;
  return (unsigned)((long long)a.B * a.blocks_t * ((a.C / E + lanes - 1) / lanes));
}

#define KDA_CONV_W(W_, CALL)      \
  switch (W_) {                   \
    case 2: { constexpr int W = 2; CALL; } break; \
    case 3: { constexpr int W = 3; CALL; } break; \
    default: { constexpr int W = 4; CALL; } break; \
  }

}  // namespace

template <typename T>
hipError_t launch_conv_fwd(const void* x, long long xb, long long xt, const float* w, const float* bias,
                           const int* lengths, const void* state_in, int silu, void* y, void* state_out, int B, int H,
                           int T_, int D, int W_, hipStream_t s) {
  ConvArgs a = {};
  a.x = x, a.xb = xb, a.xt = xt, a.w = w, a.bias = bias, a.lengths = lengths, a.state_in = state_in;
  a.y = y, a.state_out = state_out, a.B = B, a.H = H, a.T = T_, a.D = D, a.C = H * D, a.silu = silu;
  constexpr int E = conv_e<T>(false);
  conv_plan(a, E);
  KDA_CONV_W(W_, (conv_fwd_kernel<T, W, E><<<conv_grid(a, E), kConvThreads, 0, s>>>(a)))
  return hipGetLastError();
}

template <typename T>
hipError_t launch_conv_step(const void* x, long long xb, const float* w, const float* bias, int silu, void* state,
                            void* y, int B, int C, int W_, hipStream_t s) {
  ConvArgs a = {};
  a.x = x, a.xb = xb, a.w = w, a.bias = bias, a.y = y, a.state_out = state, a.B = B, a.C = C, a.silu = silu;
  constexpr int E = conv_e<T>(false);
  const unsigned grid = (unsigned)(((long long)((B + kConvStepBatch - 1) / kConvStepBatch) * (C / E) + kConvThreads - 1) / kConvThreads);
  KDA_CONV_W(W_, (conv_step_kernel<T, W, E><<<grid, kConvThreads, 0, s>>>(a)))
  return hipGetLastError();
}

size_t conv_bwd_workspace_bytes(int B, int H, int T, int D, int W, bool bf16) {
  ConvArgs a = {};
  a.B = B, a.T = T, a.C = H * D;
  conv_plan(a, bf16 ? conv_e<bf16_t>(true) : conv_e<float>(true));
  return (size_t)B * a.blocks_t * (W + 1) * a.C * 4;
}

template <typename T>
hipError_t launch_conv_bwd(const void* x, long long xb, long long xt, const float* w, const float* bias,
                           const int* lengths, const void* state_in, int silu, const void* dy, const float* d_state,
                           void* dx, long long dxb, long long dxt, float* dw, float* db, float* d_state_in,
                           void* workspace, int B, int H, int T_, int D, int W_, hipStream_t s) {
  ConvArgs a = {};
  a.x = x, a.xb = xb, a.xt = xt, a.w = w, a.bias = bias, a.lengths = lengths, a.state_in = state_in;
  a.dy = dy, a.d_state = d_state, a.dx = dx, a.db = dxb, a.dt = dxt, a.d_state_in = d_state_in;
  a.B = B, a.H = H, a.T = T_, a.D = D, a.C = H * D, a.silu = silu;
  a.parts = dw || db ? (float*)workspace : nullptr;
  constexpr int E = conv_e<T>(true);
  conv_plan(a, E);
  const int parts = B * a.blocks_t;
  if (silu) {
    KDA_CONV_W(W_, (conv_bwd_kernel<T, W, E, true><<<conv_grid(a, E), kConvThreads, 0, s>>>(a)))
  } else {
    KDA_CONV_W(W_, (conv_bwd_kernel<T, W, E, false><<<conv_grid(a, E), kConvThreads, 0, s>>>(a)))
  }
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || !a.parts) return e;
  KDA_CONV_W(W_, (conv_params_kernel<W><<<((W + 1) * a.C + 63) / 64, kSumThreads, 0, s>>>(a.parts, parts, a.C, dw, db)))
  return hipGetLastError();
}

#define KDA_CONV_INST(T)                                                                                               \
  template hipError_t launch_conv_fwd<T>(const void*, long long, long long, const float*, const float*, const int*,    \
                                         const void*, int, void*, void*, int, int, int, int, int, hipStream_t);        \
  template hipError_t launch_conv_step<T>(const void*, long long, const float*, const float*, int, void*, void*, int,  \
                                          int, int, hipStream_t);                                                      \
  template hipError_t launch_conv_bwd<T>(const void*, long long, long long, const float*, const float*, const int*,    \
                                         const void*, int, const void*, const float*, void*, long long, long long,     \
                                         float*, float*, float*, void*, int, int, int, int, int, hipStream_t);
KDA_CONV_INST(float)
KDA_CONV_INST(bf16_t)

}  // namespace kda
