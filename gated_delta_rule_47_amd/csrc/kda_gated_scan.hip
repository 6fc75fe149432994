// Gated linear recurrence, one state per channel: prompts, single tokens, adjoint.
//
//   g = -m softplus(z + dt_bias), m = exp(clamp(A_log, -10, 20)),  a = e^g,  n = (1 - a^2)^1/2 or 1,  s = sigmoid(i) or 1
//   h_t = a_t h_{t-1} + n_t s_t x_t,  y = h
//   r_t = dL/dh_t = dy_t + a_{t+1} r_{t+1}:  dx = r n s,  di = r n x s (1 - s),
//   dg = r (a h_{t-1} - a^2 / n s x),  dz = -dg m sigmoid(z + dt_bias),  dA_log = sum dg g,  ddt_bias = sum dz
#include "../../include/kda.h"
#include "kda_launch.h"
#include "kda_vec.h"

namespace kda {
namespace {

constexpr int kScanThreads = 256;
constexpr int kScanChunk = KDA_GATED_SCAN_CHUNK;

__device__ __forceinline__ float sigmoid_f(float x) { return fast_rcp(1.0f + fast_exp2(-kLog2e * x)); }

// The decay of one token.  A decay next to 1 rounded to fp32 is off to the same side in every token of a channel whose
// gate hardly moves, by up to 2^-25 / |g| of the state after the 1 / |g| tokens it remembers.  So a weak one (|g| < 1/8)
// is held as e = a - 1, a strong one as a.
struct Decay {
  float v;                                 // e or a
  bool weak;
  __device__ __forceinline__ float step(float h, float u) const { return fmaf(v, h, (weak ? h : 0.f) + u); }
  __device__ __forceinline__ float a() const { return weak ? 1.f + v : v; }
  __device__ __forceinline__ float n2() const { return weak ? -v * (2.f + v) : fmaf(-v, v, 1.f); }   // 1 - a^2
};
__device__ __forceinline__ Decay decay_of(float g2) {     // g2 = g log2(e)
  // e^g - 1 to the fifth power of g: the sixth is below 2^-27 of it at 1/8
  const float g = g2 * kLn2;
  const float e = g * fmaf(g, fmaf(g, fmaf(g, fmaf(g, 1.f / 120, 1.f / 24), 1.f / 6), 0.5f), 1.f);
  Decay d;
  d.weak = g > -0.125f;
  d.v = d.weak ? e : fast_exp2(g2);
  return d;
}

struct ScanArgs {
  const void *x, *z, *i;
  const float *A_log, *dt_bias;
  const int* lengths;
  const float* state_in;
  void* y;
  float *state_out, *ckpt;
  const void* dy;                          // backward
  const float* d_state;
  void *dx, *dz, *di;
  float *d_state_in, *parts;
  int B, H, T, D, normalize;
};

template <typename T> __global__ __launch_bounds__(kScanThreads) void scan_fwd_kernel(ScanArgs a) {
  const long long N = (long long)a.B * a.H * a.D, ch = (long long)blockIdx.x * kScanThreads + threadIdx.x;
  if (ch >= N) return;
  const int bh = (int)(ch / a.D), d = (int)(ch % a.D), h = bh % a.H, b = bh / a.H;
  const float m = gate_multiplier(a.A_log[h]), bias = a.dt_bias ? a.dt_bias[h * a.D + d] : 0.f;
  const int n = a.lengths ? min(max(a.lengths[b], 0), a.T) : a.T;
  const size_t base = (size_t)bh * a.T * a.D + d;
  const int chunks = (a.T + kScanChunk - 1) / kScanChunk;
  float st = a.state_in ? a.state_in[ch] : 0.f;
  for (int t = 0; t < a.T; ++t) {
    if (a.ckpt && t % kScanChunk == 0) a.ckpt[((size_t)bh * chunks + t / kScanChunk) * a.D + d] = st;
    if (t >= n) continue;
    const size_t o = base + (size_t)t * a.D;
    const Decay dec = decay_of(-m * softplus2_f((to_f<T>(((const T*)a.z)[o]) + bias) * kLog2e, true));
    float u = to_f<T>(((const T*)a.x)[o]);
    if (a.i) u *= sigmoid_f(to_f<T>(((const T*)a.i)[o]));
    if (a.normalize) u *= sqrtf(dec.n2());
    st = dec.step(st, u);
    ((T*)a.y)[o] = from_f<T>(st);
  }
  if (a.state_out) a.state_out[ch] = st;
}

template <typename T> __global__ __launch_bounds__(kScanThreads) void scan_bwd_kernel(ScanArgs a) {
  const long long N = (long long)a.B * a.H * a.D, ch = (long long)blockIdx.x * kScanThreads + threadIdx.x;
  if (ch >= N) return;
  const int bh = (int)(ch / a.D), d = (int)(ch % a.D), h = bh % a.H, b = bh / a.H;
  const float m = gate_multiplier(a.A_log[h]), bias = a.dt_bias ? a.dt_bias[h * a.D + d] : 0.f;
  const int n = a.lengths ? min(max(a.lengths[b], 0), a.T) : a.T;
  const size_t base = (size_t)bh * a.T * a.D + d;
  const int chunks = (a.T + kScanChunk - 1) / kScanChunk;
  float r = a.d_state ? a.d_state[ch] : 0.f, sz = 0.f, sa = 0.f;
  for (int t = n; t < a.T; ++t) {
    const size_t o = base + (size_t)t * a.D;
    ((T*)a.dx)[o] = ((T*)a.dz)[o] = from_f<T>(0.f);
    if (a.di) ((T*)a.di)[o] = from_f<T>(0.f);
  }
  for (int c = (n + kScanChunk - 1) / kScanChunk - 1; c >= 0; --c) {
    float before[kScanChunk];
    float st = a.ckpt[((size_t)bh * chunks + c) * a.D + d];
    for (int k = 0; k < kScanChunk; ++k) {
      const int t = c * kScanChunk + k;
      if (t >= n) break;
      const size_t o = base + (size_t)t * a.D;
      before[k] = st;
      const Decay dec = decay_of(-m * softplus2_f((to_f<T>(((const T*)a.z)[o]) + bias) * kLog2e, true));
      float u = to_f<T>(((const T*)a.x)[o]);
      if (a.i) u *= sigmoid_f(to_f<T>(((const T*)a.i)[o]));
      if (a.normalize) u *= sqrtf(dec.n2());
      st = dec.step(st, u);
    }
    for (int k = kScanChunk - 1; k >= 0; --k) {
      const int t = c * kScanChunk + k;
      if (t >= n) continue;
      const size_t o = base + (size_t)t * a.D;
      const float p = to_f<T>(((const T*)a.z)[o]) + bias, x = to_f<T>(((const T*)a.x)[o]);
      const float sp2 = softplus2_f(p * kLog2e, true);
      const Decay dec = decay_of(-m * sp2);
      const float s = a.i ? sigmoid_f(to_f<T>(((const T*)a.i)[o])) : 1.f;
      const float nn = fmaxf(dec.n2(), 1e-38f), rn = a.normalize ? __builtin_amdgcn_rsqf(nn) : 1.f;
      const float nrm = a.normalize ? dec.n2() * rn : 1.f, av = dec.a();
      r += to_f<T>(((const T*)a.dy)[o]);
      const float q = m * sigmoid_f(p);
      ((T*)a.dx)[o] = from_f<T>(r * nrm * s);
      if (a.di) ((T*)a.di)[o] = from_f<T>(r * nrm * x * s * (1.f - s));
      float w = av * before[k] * q;
      if (a.normalize) w -= q * av * av * s * x * rn;
      ((T*)a.dz)[o] = from_f<T>(-r * w);
      sz -= r * w;
      float dg = av * before[k];
      if (a.normalize) dg -= av * av * s * x * rn;
      sa += r * dg * (-m * sp2 * kLn2);
      r = dec.step(r, 0.f);
    }
  }
  a.d_state_in[ch] = r;
  a.parts[ch] = sz;
  a.parts[N + ch] = sa;
}

__global__ void scan_params_kernel(ScanArgs a, float* dA_log, float* d_dt_bias) {
  const long long N = (long long)a.B * a.H * a.D;
  const int hd = a.H * a.D;
  for (int k = blockIdx.x * blockDim.x + threadIdx.x; k < hd; k += gridDim.x * blockDim.x) {
    float s = 0.f;
    for (int b = 0; b < a.B; ++b) s += a.parts[(size_t)b * hd + k];
    if (d_dt_bias) d_dt_bias[k] = s;
  }
  for (int h = blockIdx.x * blockDim.x + threadIdx.x; h < a.H; h += gridDim.x * blockDim.x) {
    float s = 0.f;
    for (int b = 0; b < a.B; ++b)
      for (int d = 0; d < a.D; ++d) s += a.parts[N + ((size_t)b * a.H + h) * a.D + d];
    if (dA_log) dA_log[h] = a.A_log[h] >= kALogMin && a.A_log[h] <= kALogMax ? s : 0.f;
  }
}

template <typename T> __global__ __launch_bounds__(kScanThreads) void scan_step_kernel(ScanArgs a) {
  const long long N = (long long)a.B * a.H * a.D, ch = (long long)blockIdx.x * kScanThreads + threadIdx.x;
  if (ch >= N) return;
  const int d = (int)(ch % a.D), h = (int)(ch / a.D % a.H);
  const float m = gate_multiplier(a.A_log[h]), bias = a.dt_bias ? a.dt_bias[h * a.D + d] : 0.f;
  const Decay dec = decay_of(-m * softplus2_f((to_f<T>(((const T*)a.z)[ch]) + bias) * kLog2e, true));
  float u = to_f<T>(((const T*)a.x)[ch]);
  if (a.i) u *= sigmoid_f(to_f<T>(((const T*)a.i)[ch]));
  if (a.normalize) u *= sqrtf(dec.n2());
  const float st = dec.step(a.state_out[ch], u);
  a.state_out[ch] = st;
  ((T*)a.y)[ch] = from_f<T>(st);
}

unsigned scan_grid(const ScanArgs& a) {
  return (unsigned)(((long long)a.B * a.H * a.D + kScanThreads - 1) / kScanThreads);
}

ScanArgs scan_args(const void* x, const void* z, const float* A_log, const float* dt_bias, const void* i,
                   const int* lengths, int normalize, int B, int H, int T, int D) {
  ScanArgs a = {};
  a.x = x, a.z = z, a.A_log = A_log, a.dt_bias = dt_bias, a.i = i, a.lengths = lengths, a.normalize = normalize;
  a.B = B, a.H = H, a.T = T, a.D = D;
  return a;
}

}  // namespace

size_t scan_workspace_bytes(int, int, int, int, bool) { return 0; }
size_t scan_bwd_workspace_bytes(int B, int H, int, int D, bool) { return (size_t)B * H * D * 8; }

template <typename T>
hipError_t launch_scan_fwd(const void* x, const void* z, const float* A_log, const float* dt_bias, const void* i,
                           const int* lengths, const float* state_in, int normalize, void* y, float* state_out,
                           float* ckpt, void*, int B, int H, int T_, int D, hipStream_t s) {
  ScanArgs a = scan_args(x, z, A_log, dt_bias, i, lengths, normalize, B, H, T_, D);
  a.state_in = state_in, a.y = y, a.state_out = state_out, a.ckpt = ckpt;
  scan_fwd_kernel<T><<<scan_grid(a), kScanThreads, 0, s>>>(a);
  return hipGetLastError();
}

template <typename T>
hipError_t launch_scan_step(const void* x, const void* z, const float* A_log, const float* dt_bias, const void* i,
                            int normalize, float* state, void* y, int B, int H, int D, hipStream_t s) {
  ScanArgs a = scan_args(x, z, A_log, dt_bias, i, nullptr, normalize, B, H, 1, D);
  a.state_out = state, a.y = y;
  scan_step_kernel<T><<<scan_grid(a), kScanThreads, 0, s>>>(a);
  return hipGetLastError();
}

template <typename T>
hipError_t launch_scan_bwd(const void* x, const void* z, const float* A_log, const float* dt_bias, const void* i,
                           const int* lengths, int normalize, const float* ckpt, const void* dy, const float* d_state,
                           void* dx, void* dz, void* di, float* dA_log, float* d_dt_bias, float* d_state_in,
                           void* workspace, int B, int H, int T_, int D, hipStream_t s) {
  ScanArgs a = scan_args(x, z, A_log, dt_bias, i, lengths, normalize, B, H, T_, D);
  a.ckpt = const_cast<float*>(ckpt), a.dy = dy, a.d_state = d_state, a.dx = dx, a.dz = dz, a.di = di;
  a.d_state_in = d_state_in, a.parts = (float*)workspace;
  scan_bwd_kernel<T><<<scan_grid(a), kScanThreads, 0, s>>>(a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  scan_params_kernel<<<64, kScanThreads, 0, s>>>(a, dA_log, d_dt_bias);
  return hipGetLastError();
}

#define KDA_SCAN_INST(T)                                                                                               \
  template hipError_t launch_scan_fwd<T>(const void*, const void*, const float*, const float*, const void*, const int*, \
                                         const float*, int, void*, float*, float*, void*, int, int, int, int,          \
                                         hipStream_t);                                                                 \
  template hipError_t launch_scan_step<T>(const void*, const void*, const float*, const float*, const void*, int,      \
                                          float*, void*, int, int, int, hipStream_t);                                  \
  template hipError_t launch_scan_bwd<T>(const void*, const void*, const float*, const float*, const void*, const int*, \
                                         int, const float*, const void*, const float*, void*, void*, void*, float*,    \
                                         float*, float*, void*, int, int, int, int, hipStream_t);
KDA_SCAN_INST(float)
KDA_SCAN_INST(bf16_t)

}  // namespace kda
