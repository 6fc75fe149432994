// Host side of the gated recurrence, its single token, and the small kernels around the tiles (kda_gated_scan.h).
#include "kda_gated_scan.h"

namespace kda {
namespace {

constexpr int kScanThreads = 256;

// Clears the counters and the flags (a kernel, not a memset: it may be captured into a graph).
__global__ __launch_bounds__(kScanThreads) void scan_clear_kernel(uint32_t* p, uint32_t n) {
  const uint32_t i = blockIdx.x * kScanThreads + threadIdx.x;
  if (i < n) p[i] = 0u;
}

// ddt_bias, and the sums of dg g over time and sequences, from the tiles' parts.
__global__ __launch_bounds__(kSumThreads) void scan_params_kernel(const float* parts, size_t half, int n_parts, int n,
                                                                  float* d_dt_bias, float* sums) {
  float* out = blockIdx.y ? sums : d_dt_bias;
  if (!out) return;
  sum_parts(parts + blockIdx.y * half, n, n_parts, n, [=](int i, float s) { out[i] = s; });
}
// dA_log of head h: the sum of n_parts rows of its D channels, `stride` apart, in a fixed order.
__device__ __forceinline__ void scan_head_sum(const float* in, size_t stride, int n_parts, const float* A_log, int D, int h,
                                              float* dA_log) {
  __shared__ float red[kSumThreads / 64];
  const float* p = in + (size_t)h * D;
  const uint32_t q = kSumThreads / (uint32_t)D, r = kSumThreads % (uint32_t)D;       // rows and channels from value to value
  uint32_t row = threadIdx.x / (uint32_t)D, col = threadIdx.x % (uint32_t)D;
  float s = 0.f;
#pragma unroll 8
  while (row < (uint32_t)n_parts) {
    s += p[(size_t)row * stride + col];
    row += q;
    col += r;
    if (col >= (uint32_t)D) col -= (uint32_t)D, ++row;
  }
  s = lane_sum<64>(s);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x == 0) {
    s = 0.f;
    for (int k = 0; k < kSumThreads / 64; ++k) s += red[k];
    const float al = A_log[h];
    dA_log[h] = al < kALogMin || al > kALogMax ? 0.f : s;              // the clamp holds the multiplier constant there
  }
}
__global__ __launch_bounds__(kSumThreads) void scan_head_kernel(const float* sums, const float* A_log, int D, float* dA_log) {
  scan_head_sum(sums, 0, 1, A_log, D, blockIdx.x, dA_log);
}
// Both in one launch where a head has few values: first the workgroups of ddt_bias, then one per head.
__global__ __launch_bounds__(kSumThreads) void scan_small_params_kernel(const float* parts, size_t half, int n_parts, int n,
                                                                        const float* A_log, int D, float* d_dt_bias, float* dA_log) {
  const int blocks = (n + 63) / 64, b = blockIdx.x;
  if (b < blocks) {
    if (d_dt_bias) sum_parts(parts, n, n_parts, n, [=](int i, float s) { d_dt_bias[i] = s; });
  } else if (dA_log) {
    scan_head_sum(parts + half, n, n_parts, A_log, D, b - blocks, dA_log);
  }
}

// One token: bound by launch and memory latency; a lane takes E neighbouring channels.
template <typename T, int E> __global__ __launch_bounds__(kScanThreads) void scan_step_kernel(ScanArgs a) {
  const uint32_t ch = (blockIdx.x * kScanThreads + threadIdx.x) * E;
  if (ch >= (uint32_t)(a.B * a.H * a.D)) return;
  const uint32_t row = ch / (uint32_t)a.D, d = ch - row * (uint32_t)a.D, h = row % (uint32_t)a.H;
  const uint32_t off = ch * sizeof(T);     // B H D <= 2^26
  ScanRaw<T, E> rz, rx, ri;
  rz.load(a.z, off);
  rx.load(a.x, off);
  if (a.i) ri.load(a.i, off);
  const float m = gate_multiplier(a.A_log[h]);
  float st[E];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    float y, u = rx.at(e);
    const float bias2 = a.dt_bias ? a.dt_bias[(size_t)h * a.D + d + e] * kLog2e : 0.f;
    const float v = decay_of(-m * scan_softplus2(fmaf(rz.at(e), kLog2e, bias2), y));
    if (a.i) u *= scan_sigmoid(ri.at(e));
    if (a.normalize) u *= __builtin_amdgcn_sqrtf(decay_n2(v));
    st[e] = decay_step(v, a.state_out[ch + e], u);
    a.state_out[ch + e] = st[e];
  }
  scan_store<T, E>(a.y, off, st);
}

ScanArgs scan_args(const void* x, const void* z, const float* A_log, const float* dt_bias, const void* i,
                   const int* lengths, int normalize, int B, int H, int T, int D) {
  ScanArgs a = {};
  a.x = x, a.z = z, a.A_log = A_log, a.dt_bias = dt_bias, a.i = i, a.lengths = lengths, a.normalize = normalize;
  a.B = B, a.H = H, a.T = T, a.D = D;
  return a;
}

// Channels per lane: two bf16, for one token only where no head's end separates them.
int scan_e(int D, bool bf16) { return bf16 && D > 1 ? 2 : 1; }
int scan_step_e(int D, bool bf16) { return bf16 && D % 2 == 0 ? 2 : 1; }

struct ScanPlan {
  int E, ctiles, tiles, groups;
  size_t every, flags, group_flags, clear, pairs, states, group_pairs, parts, sums, total;   // words per counter; offsets and the bytes cleared
};
size_t up(size_t n) { return (n + 255) / 256 * 256; }
ScanPlan scan_plan(int B, int H, int T, int D, bool bf16, bool bwd) {
  ScanPlan p;
  const long long N = (long long)B * H * D;
  p.E = scan_e(D, bf16);
  p.ctiles = (int)(((long long)B * H * ((D + p.E - 1) / p.E) + 63) / 64);
  const int tokens = bwd ? scan_bwd_waves(p.ctiles) * kScanBwdTokens : scan_fwd_waves(p.ctiles) * kScanFwdTokens;
  p.tiles = T > tokens ? (T + tokens - 1) / tokens : 1;
  const size_t n = p.tiles > 1 ? (size_t)p.ctiles * p.tiles : 0;
  p.every = p.ctiles <= 4096 ? 32 : 1;
  p.flags = up(n ? p.every * p.ctiles * 4 : 0);
  p.groups = scan_grouped(p.ctiles, p.tiles) ? (p.tiles >> kScanGroupLog2) + 1 : 0;
  const size_t ng = (size_t)p.ctiles * p.groups;
  p.group_flags = p.flags + n * 4;
  p.clear = p.group_flags + ng * 4;
  p.pairs = up(p.clear);
  p.states = p.pairs + n * 128 * p.E * 4;
  p.group_pairs = p.states + n * 64 * p.E * 4;
  p.parts = p.group_pairs + ng * 128 * p.E * 4;
  p.sums = p.parts + (bwd ? up((size_t)p.tiles * N * 8) : 0);
  p.total = p.sums + (bwd ? (size_t)H * D * 4 : 0);
  return p;
}
void scan_link(ScanArgs& a, const ScanPlan& p, void* workspace, hipStream_t s) {
  char* w = (char*)workspace;
  a.ctiles = p.ctiles, a.tiles = p.tiles;
  if (!p.clear) return;
  a.link.tickets = (uint32_t*)w, a.link.flags = (uint32_t*)(w + p.flags), a.link.every = (uint32_t)p.every;
  a.link.pairs = (float*)(w + p.pairs), a.link.states = (float*)(w + p.states);
  a.link.group_flags = (uint32_t*)(w + p.group_flags), a.link.group_pairs = (float*)(w + p.group_pairs);
  a.link.groups = (uint32_t)p.groups;
  const uint32_t n = (uint32_t)(p.clear / 4);
  scan_clear_kernel<<<(n + kScanThreads - 1) / kScanThreads, kScanThreads, 0, s>>>((uint32_t*)w, n);
}

}  // namespace

size_t scan_workspace_bytes(int B, int H, int T, int D, bool bf16) { return scan_plan(B, H, T, D, bf16, false).total; }
size_t scan_bwd_workspace_bytes(int B, int H, int T, int D, bool bf16) { return scan_plan(B, H, T, D, bf16, true).total; }

template <typename T>
hipError_t launch_scan_fwd(const void* x, const void* z, const float* A_log, const float* dt_bias, const void* i,
                           const int* lengths, const float* state_in, int normalize, void* y, float* state_out,
                           float* ckpt, void* workspace, int B, int H, int T_, int D, hipStream_t s) {
  ScanArgs a = scan_args(x, z, A_log, dt_bias, i, lengths, normalize, B, H, T_, D);
  a.state_in = state_in, a.y = y, a.state_out = state_out, a.ckpt = ckpt;
  const ScanPlan p = scan_plan(B, H, T_, D, sizeof(T) == 2, false);
  scan_link(a, p, workspace, s);
  return launch_scan_fwd_tiles<T>(a, p.E == 2, s);
}

template <typename T>
hipError_t launch_scan_step(const void* x, const void* z, const float* A_log, const float* dt_bias, const void* i,
                            int normalize, float* state, void* y, int B, int H, int D, hipStream_t s) {
  ScanArgs a = scan_args(x, z, A_log, dt_bias, i, nullptr, normalize, B, H, 1, D);
  a.state_out = state, a.y = y;
  const int E = scan_step_e(D, sizeof(T) == 2);
  const unsigned grid = (unsigned)(((long long)B * H * D / E + kScanThreads - 1) / kScanThreads);
  if constexpr (sizeof(T) == 2)
    if (E == 2) {
      scan_step_kernel<T, 2><<<grid, kScanThreads, 0, s>>>(a);
      return hipGetLastError();
    }
  scan_step_kernel<T, 1><<<grid, kScanThreads, 0, s>>>(a);
  return hipGetLastError();
}

template <typename T>
hipError_t launch_scan_bwd(const void* x, const void* z, const float* A_log, const float* dt_bias, const void* i,
                           const int* lengths, int normalize, const float* ckpt, const void* dy, const float* d_state,
                           void* dx, void* dz, void* di, float* dA_log, float* d_dt_bias, float* d_state_in,
                           void* workspace, int B, int H, int T_, int D, hipStream_t s) {
  ScanArgs a = scan_args(x, z, A_log, dt_bias, i, lengths, normalize, B, H, T_, D);
  a.ckpt = const_cast<float*>(ckpt), a.dy = dy, a.d_state = d_state, a.dx = dx, a.dz = dz, a.di = di;
  a.d_state_in = d_state_in;
  const ScanPlan p = scan_plan(B, H, T_, D, sizeof(T) == 2, true);
  float* sums = (float*)((char*)workspace + p.sums);
  if (dA_log || d_dt_bias) a.parts = (float*)((char*)workspace + p.parts);
  scan_link(a, p, workspace, s);
  hipError_t e = launch_scan_bwd_tiles<T>(a, p.E == 2, s);
  if (e != hipSuccess || !a.parts) return e;
  const int n = H * D;
  // up to 8 values per thread of a head's workgroup (2048 x 256: 21.0 us the whole adjoint, 20.7 in two launches); beyond, the
  // channels are summed over time first, by many workgroups (2048 x 512: 21.3 us, 23.7 in one launch; 4096 x 1024: 33 and 50).
  // Few channels of many sequences leave all parts to two workgroups: 16 x 32768 x 8, bf16, 27 us of the step's 102.
  if ((long long)p.tiles * B * D <= 8 * kSumThreads) {
    scan_small_params_kernel<<<(n + 63) / 64 + H, kSumThreads, 0, s>>>(a.parts, (size_t)p.tiles * B * n, p.tiles * B, n, A_log, D,
                                                                       d_dt_bias, dA_log);
    return hipGetLastError();
  }
  scan_params_kernel<<<dim3((n + 63) / 64, 2), kSumThreads, 0, s>>>(a.parts, (size_t)p.tiles * B * n, p.tiles * B, n,
                                                                    d_dt_bias, dA_log ? sums : nullptr);
  e = hipGetLastError();
  if (e != hipSuccess || !dA_log) return e;
  scan_head_kernel<<<H, kSumThreads, 0, s>>>(sums, A_log, D, dA_log);
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
