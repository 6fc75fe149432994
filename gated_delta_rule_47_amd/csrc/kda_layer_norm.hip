// Layer norm over the last axis of (B, H, T, D) with a weight and bias row per head, forward and
// backward.
//
//   mean = sum x / D, rstd = (sum (x - mean)^2 / D + eps)^-1/2, y = (x - mean) rstd w + b
//   xh = (x - mean) rstd, p = dy w, dx = rstd (p - mean(p) - xh mean(p xh))
//   dw = sum over the head's rows of dy xh, db = sum of dy
//
// Both are bound by memory: one read of each input, one write.  A row is held in the registers of L
// lanes (16 bytes per lane and vector, NV vectors), so the statistics take two passes over registers,
// not memory.  A workgroup takes a run of rows of one head, so that the head's weights are read once
// into registers and the weight's gradient is summed in registers over the run; the runs' sums are
// added in a fixed order by a second kernel (repeatable bit by bit, no atomics).
#include <type_traits>

#include "kda_decay_attn.h"
#include "kda_launch.h"

namespace kda {

constexpr int kNormThreads = 256;

// Sum over the L lanes of a row: a power of two up to 64, or the whole workgroup (whose four waves add
// in a fixed order through `red`); every lane of the row gets it.
template <int L> __device__ __forceinline__ float row_sum(float x, float* red) {
#pragma unroll
  for (int m = 1; m < (L < 64 ? L : 64); m <<= 1) x += __shfl_xor(x, m, 64);
  if constexpr (L > 64) {
    static_assert(L == kNormThreads, "rows of a wave or of the workgroup");
    __syncthreads();
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = x;
    __syncthreads();
    x = (red[0] + red[1]) + (red[2] + red[3]);
  }
  return x;
}

// E consecutive elements of a row in fp32: 16 bytes of T (Wide<T>::E of them), or one element where the
// width or an address keeps rows from being 16-byte aligned.
template <typename T> struct Wide {
  static constexpr int E = 16 / (int)sizeof(T);
};
template <typename T, int E> __device__ __forceinline__ void vec_get(const T* p, float* f) {
  if constexpr (E == 1) {
    f[0] = to_f<T>(*p);
  } else {
    const u32x4_t u = *reinterpret_cast<const u32x4_t*>(p);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (E == 4) {
        f[i] = __uint_as_float(u[i]);
      } else {
        f[2 * i] = __uint_as_float(u[i] << 16);
        f[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
      }
    }
  }
}
template <typename T, int E> __device__ __forceinline__ void vec_put(T* p, const float* f) {
  if constexpr (E == 1) {
    *p = from_f<T>(f[0]);
  } else {
    u32x4_t u;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (E == 4) u[i] = __float_as_uint(f[i]);
      else u[i] = pack_bf16x2(f[2 * i], f[2 * i + 1]);
    }
    *reinterpret_cast<u32x4_t*>(p) = u;
  }
}
// E codes of an 8-bit tensor with the scale s
template <int E> __device__ __forceinline__ void vec_codes(const uint8_t* p, float s, float* f) {
  if constexpr (E == 1) {
    f[0] = __builtin_amdgcn_cvt_pk_f32_fp8((int)*p, false)[0] * s;
  } else {
#pragma unroll
    for (int i = 0; i < E / 4; ++i) {
      const uint32_t u = reinterpret_cast<const uint32_t*>(p)[i];
      const floatx2 a = __builtin_amdgcn_cvt_pk_f32_fp8((int)u, false);
      const floatx2 b = __builtin_amdgcn_cvt_pk_f32_fp8((int)u, true);
      f[4 * i] = a[0] * s;
      f[4 * i + 1] = a[1] * s;
      f[4 * i + 2] = b[0] * s;
      f[4 * i + 3] = b[1] * s;
    }
  }
}

// Value i of an 8-bit tensor with D channels, one scale byte per `grp` channels.
__device__ __forceinline__ float ckpt_value(const uint8_t* codes, const uint8_t* sc, size_t row, int i, int D,
                                            int grp) {
  const floatx2 a = __builtin_amdgcn_cvt_pk_f32_fp8((int)codes[row * D + i], false);
  return a[0] * ckpt_scale(sc[row * (D / grp) + i / grp]);
}

// (var + eps)^-1/2; a variance that rounding left below zero is zero, NaN stays NaN
__device__ __forceinline__ float rstd_of(float var, float eps) { return 1.0f / sqrtf((var < 0.0f ? 0.0f : var) + eps); }

// ------------------------------------------------------------------ forward
template <typename T, int E, int L, int NV>
__global__ void __launch_bounds__(kNormThreads) norm_fwd_kernel(const T* __restrict__ x, const float* __restrict__ w,
                                                                const float* __restrict__ b, float eps,
                                                                T* __restrict__ y, float* __restrict__ mean,
                                                                float* __restrict__ rstd, int H, int T_, int D,
                                                                int ntile, int tile_rows) {
  constexpr int RPW = kNormThreads / L;
  __shared__ float rsum[kNormThreads / 64];
  const int bh = blockIdx.x / ntile, tile = blockIdx.x - bh * ntile;
  const int c = threadIdx.x % L, rr = threadIdx.x / L;
  const float inv = 1.0f / (float)D;
  float wv[NV][E], bv[NV][E];
  bool in[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int col = (c + i * L) * E;
    in[i] = col < D;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      wv[i][e] = in[i] && w ? w[(size_t)(bh % H) * D + col + e] : 1.0f;
      bv[i][e] = in[i] && b ? b[(size_t)(bh % H) * D + col + e] : 0.0f;
    }
  }
  const int t_end = min(T_, (tile + 1) * tile_rows);
  for (int t = tile * tile_rows + rr; t < t_end; t += RPW) {
    const size_t row = (size_t)bh * T_ + t;
    float v[NV][E];
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (in[i]) vec_get<T, E>(x + row * D + (c + i * L) * E, v[i]);
#pragma unroll
      for (int e = 0; e < E; ++e) s += in[i] ? v[i][e] : 0.0f;
    }
    const float m = row_sum<L>(s, rsum) * inv;
    float q = 0.0f, d = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < E; ++e) {
        v[i][e] -= m;
        q += in[i] ? v[i][e] * v[i][e] : 0.0f;
        d += in[i] ? v[i][e] : 0.0f;
      }
    // m is rounded (by up to 2^-24 |m|, which shows where a row's mean is far above its spread): what is
    // left of the mean in the differences is taken out of them and of their squares
    const float dm = row_sum<L>(d, rsum) * inv;
    const float r = rstd_of(row_sum<L>(q, rsum) * inv - dm * dm, eps);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
#pragma unroll
      for (int e = 0; e < E; ++e) v[i][e] = fmaf((v[i][e] - dm) * r, wv[i][e], bv[i][e]);
      if (in[i]) vec_put<T, E>(y + row * D + (c + i * L) * E, v[i]);
    }
    if (c == 0) {
      if (mean) mean[row] = m + dm;
      if (rstd) rstd[row] = r;
    }
  }
}

// Any width and alignment: a workgroup per row, which is read three times (the second and third time
// from cache for rows that fit it).
template <typename T>
__global__ void __launch_bounds__(kNormThreads) norm_fwd_any_kernel(const T* __restrict__ x,
                                                                    const float* __restrict__ w,
                                                                    const float* __restrict__ b, float eps,
                                                                    T* __restrict__ y, float* __restrict__ mean,
                                                                    float* __restrict__ rstd, int H, int T_, int D) {
  __shared__ float red[kNormThreads / 64];
  const size_t row = blockIdx.x;
  const int h = (int)(row / T_ % H);
  const T* xr = x + row * D;
  float s = 0.0f;
  for (int i = threadIdx.x; i < D; i += kNormThreads) s += to_f<T>(xr[i]);
  const float m = row_sum<kNormThreads>(s, red) / (float)D;
  float q = 0.0f, sd = 0.0f;
  for (int i = threadIdx.x; i < D; i += kNormThreads) {
    const float d = to_f<T>(xr[i]) - m;
    q += d * d;
    sd += d;
  }
  const float dm = row_sum<kNormThreads>(sd, red) / (float)D;     // the rounding of m, as above
  const float r = rstd_of(row_sum<kNormThreads>(q, red) / (float)D - dm * dm, eps);
  for (int i = threadIdx.x; i < D; i += kNormThreads) {
    const float wi = w ? w[(size_t)h * D + i] : 1.0f, bi = b ? b[(size_t)h * D + i] : 0.0f;
    y[row * D + i] = from_f<T>(fmaf((to_f<T>(xr[i]) - m - dm) * r, wi, bi));
  }
  if (threadIdx.x == 0) {
    if (mean) mean[row] = m + dm;
    if (rstd) rstd[row] = r;
  }
}

// ------------------------------------------------------------------ backward
template <typename T, int E, int L, int NV, bool PK>
__global__ void __launch_bounds__(kNormThreads)
    norm_bwd_kernel(const T* __restrict__ x, const uint8_t* __restrict__ xc, const uint8_t* __restrict__ xs,
                    const float* __restrict__ w, const float* __restrict__ mean, const float* __restrict__ rstd,
                    const T* __restrict__ dy, T* __restrict__ dx, float* __restrict__ part, int H, int T_, int D,
                    int grp, int ntile, int tile_rows) {
  constexpr int RPW = kNormThreads / L;
  __shared__ float rsum[kNormThreads / 64];
  const int bh = blockIdx.x / ntile, tile = blockIdx.x - bh * ntile;
  const int c = threadIdx.x % L, rr = threadIdx.x / L;
  const float inv = 1.0f / (float)D;
  float wv[NV][E], dw[NV][E], db[NV][E];
  bool in[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int col = (c + i * L) * E;
    in[i] = col < D;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      wv[i][e] = in[i] && w ? w[(size_t)(bh % H) * D + col + e] : 1.0f;
      dw[i][e] = db[i][e] = 0.0f;
    }
  }
  const int t_end = min(T_, (tile + 1) * tile_rows);
  for (int t = tile * tile_rows + rr; t < t_end; t += RPW) {
    const size_t row = (size_t)bh * T_ + t;
    const float m = mean[row], r = rstd[row];
    float xh[NV][E], g[NV][E];
    float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int col = (c + i * L) * E;
      if (in[i]) {
        vec_get<T, E>(dy + row * D + col, g[i]);
        if constexpr (PK)
          vec_codes<E>(xc + row * D + col, ckpt_scale(xs[row * (D / grp) + col / grp]), xh[i]);
        else
          vec_get<T, E>(x + row * D + col, xh[i]);
#pragma unroll
        for (int e = 0; e < E; ++e) {
          xh[i][e] = (xh[i][e] - m) * r;
          dw[i][e] = fmaf(g[i][e], xh[i][e], dw[i][e]);
          db[i][e] += g[i][e];
          g[i][e] *= wv[i][e];
          s1 += g[i][e];
          s2 = fmaf(g[i][e], xh[i][e], s2);
        }
      }
    }
    const float c1 = row_sum<L>(s1, rsum) * inv, c2 = row_sum<L>(s2, rsum) * inv;
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (in[i]) {
#pragma unroll
        for (int e = 0; e < E; ++e) g[i][e] = r * (g[i][e] - c1 - xh[i][e] * c2);
        vec_put<T, E>(dx + row * D + (c + i * L) * E, g[i]);
      }
  }
  if (!part) return;
  // the RPW row groups of the workgroup hold sums of the same columns
  __shared__ float red[kNormThreads * E];
  float* out = part + (size_t)blockIdx.x * 2 * D;
#pragma unroll
  for (int k = 0; k < 2; ++k)
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      __syncthreads();
#pragma unroll
      for (int e = 0; e < E; ++e) red[(rr * L + c) * E + e] = k ? db[i][e] : dw[i][e];
      __syncthreads();
      for (int j = threadIdx.x; j < L * E; j += kNormThreads) {
        const int col = i * L * E + j;
        if (col < D) {
          float s = 0.0f;
          for (int g = 0; g < RPW; ++g) s += red[g * L * E + j];
          out[k * D + col] = s;
        }
      }
    }
}

// Any width and alignment: a workgroup takes the tile's rows one after another; a thread's columns
// (threadIdx.x + 256 i) keep their running sums in the workgroup's part of `part`.
template <typename T, bool PK>
__global__ void __launch_bounds__(kNormThreads)
    norm_bwd_any_kernel(const T* __restrict__ x, const uint8_t* __restrict__ xc, const uint8_t* __restrict__ xs,
                        const float* __restrict__ w, const float* __restrict__ mean, const float* __restrict__ rstd,
                        const T* __restrict__ dy, T* __restrict__ dx, float* part, int H, int T_, int D, int grp,
                        int ntile, int tile_rows) {
  __shared__ float red[kNormThreads / 64];
  const int bh = blockIdx.x / ntile, tile = blockIdx.x - bh * ntile;
  const float* wr = w ? w + (size_t)(bh % H) * D : nullptr;
  float* out = part ? part + (size_t)blockIdx.x * 2 * D : nullptr;
  const int t_beg = tile * tile_rows, t_end = min(T_, (tile + 1) * tile_rows);
  for (int t = t_beg; t < t_end; ++t) {
    const size_t row = (size_t)bh * T_ + t;
    const float m = mean[row], r = rstd[row];
    const auto xhat = [&](int i) {
      const float xv = PK ? ckpt_value(xc, xs, row, i, D, grp) : to_f<T>(x[row * D + i]);
      return (xv - m) * r;
    };
    float s1 = 0.0f, s2 = 0.0f;
    for (int i = threadIdx.x; i < D; i += kNormThreads) {
      const float d = to_f<T>(dy[row * D + i]), xh = xhat(i), p = d * (wr ? wr[i] : 1.0f);
      s1 += p;
      s2 = fmaf(p, xh, s2);
      if (out) {
        out[i] = (t == t_beg ? 0.0f : out[i]) + d * xh;
        out[D + i] = (t == t_beg ? 0.0f : out[D + i]) + d;
      }
    }
    const float c1 = row_sum<kNormThreads>(s1, red) / (float)D, c2 = row_sum<kNormThreads>(s2, red) / (float)D;
    for (int i = threadIdx.x; i < D; i += kNormThreads) {
      const float p = to_f<T>(dy[row * D + i]) * (wr ? wr[i] : 1.0f);
      dx[row * D + i] = from_f<T>(r * (p - c1 - xhat(i) * c2));
    }
  }
}

// dw[h, i], db[h, i]: sums of the parts of head h's workgroups (B * ntile of them), 64 columns per
// workgroup, four threads per column over interleaved parts.
__global__ void __launch_bounds__(256) norm_bwd_reduce_kernel(const float* __restrict__ part, float* __restrict__ dw,
                                                              float* __restrict__ db, int B, int H, int D, int ntile,
                                                              int ncol) {
  __shared__ float red[4][64];
  const int h = blockIdx.x / ncol, c0 = (blockIdx.x - h * ncol) * 64;
  const int c = c0 + (threadIdx.x & 63), sl = threadIdx.x >> 6;       // columns of dw, then of db
  float s = 0.0f;
  if (c < 2 * D)
    for (int p = sl; p < B * ntile; p += 4) {
      const int b = p / ntile, t = p - b * ntile;
      s += part[((size_t)(b * H + h) * ntile + t) * 2 * D + c];
    }
  red[sl][threadIdx.x & 63] = s;
  __syncthreads();
  if (sl == 0 && c < 2 * D) {
    s = (red[0][threadIdx.x] + red[1][threadIdx.x]) + (red[2][threadIdx.x] + red[3][threadIdx.x]);
    if (c < D) {
      if (dw) dw[(size_t)h * D + c] = s;
    } else if (db) {
      db[(size_t)h * D + c - D] = s;
    }
  }
}

// ------------------------------------------------------------------ launchers
// Rows of one workgroup: enough for the weights' read and the partial sums to be a small part of the
// rows' bytes, few enough for some 2048 workgroups (8 per CU).
struct NormPlan {
  int ntile, rows;
};
static NormPlan norm_plan(int B, int H, int T, int rpw) {
  const long long bh = (long long)B * H;
  long long tiles = (2048 + bh - 1) / bh;
  const long long most = (T + 4LL * rpw - 1) / (4LL * rpw);  // at least four steps of a workgroup's rows
  if (tiles > most) tiles = most;
  if (tiles < 1) tiles = 1;
  long long rows = (T + tiles - 1) / tiles;
  rows = (rows + rpw - 1) / rpw * rpw;
  if (rows < 1) rows = 1;
  return NormPlan{(int)((T + rows - 1) / rows), (int)rows};
}

// How a row of D elements is held: E per access, L lanes, NV accesses per lane.  One element per access
// (a quarter to an eighth of the bytes per instruction) where a row's start is not 16-byte aligned; the
// workgroup shares a row once one wave would need more than 64 (128 for 16-byte accesses) fp32
// registers for it.  NV = 0: wider than that, the any-width kernels run.
struct NormShape {
  int E, L, NV;
};
static NormShape norm_shape(int D, int Ew, bool aligned) {
  const int E = aligned && D % Ew == 0 ? Ew : 1;
  const int n = (D + E - 1) / E, wave_nv = E == 1 ? 16 : (E == 4 ? 8 : 4);
  NormShape p{E, 1, 1};
  if (E == 1) p.L = 8;
  while (p.L < n && p.L < 64) p.L <<= 1;
  while (p.NV * p.L < n) p.NV <<= 1;
  if (p.NV > wave_nv) {
    p.L = kNormThreads;
    p.NV = E == 1 ? 8 : (E == 4 ? 4 : 2);
    while (p.NV * p.L < n) p.NV <<= 1;
    if (p.NV > (E == 1 ? 32 : 8)) p.NV = 0;
  }
  return p;
}
static bool aligned16(const void* a, const void* b, const void* c) {
  return (((uintptr_t)a | (uintptr_t)b | (uintptr_t)c) & 15) == 0;
}
// The shapes above as instances: CASE(E, L, NV).
#define KDA_NORM_SHAPES(W, CASE)                                                                                   \
  CASE(W, 1, 1) CASE(W, 2, 1) CASE(W, 4, 1) CASE(W, 8, 1) CASE(W, 16, 1) CASE(W, 32, 1) CASE(W, 64, 1)             \
  CASE(W, 64, 2) CASE(W, 64, 4) CASE(W, 64, 8) CASE(W, 256, 2) CASE(W, 256, 4) CASE(W, 256, 8)                     \
  CASE(1, 8, 1) CASE(1, 16, 1) CASE(1, 32, 1) CASE(1, 64, 1) CASE(1, 64, 2) CASE(1, 64, 4) CASE(1, 64, 8)          \
  CASE(1, 64, 16) CASE(1, 256, 8) CASE(1, 256, 16) CASE(1, 256, 32)

template <typename T>
hipError_t launch_norm_fwd(const void* x, const float* w, const float* b, float eps, void* y, float* mean, float* rstd,
                           int B, int H, int T_, int D, hipStream_t s) {
  if (T_ == 0) return hipSuccess;
  const NormShape n = norm_shape(D, Wide<T>::E, aligned16(x, y, nullptr));
  if (n.NV == 0) {
    hipLaunchKernelGGL(norm_fwd_any_kernel<T>, dim3((unsigned)((size_t)B * H * T_)), dim3(kNormThreads), 0, s,
                       (const T*)x, w, b, eps, (T*)y, mean, rstd, H, T_, D);
    return hipGetLastError();
  }
  const NormPlan p = norm_plan(B, H, T_, kNormThreads / n.L);
  const dim3 grid((unsigned)(B * H * p.ntile));
#define KDA_NORM(E_, L_, NV_)                                                                                         \
  if (n.E == E_ && n.L == L_ && n.NV == NV_)                                                                          \
    hipLaunchKernelGGL((norm_fwd_kernel<T, E_, L_, NV_>), grid, dim3(kNormThreads), 0, s, (const T*)x, w, b, eps,     \
                       (T*)y, mean, rstd, H, T_, D, p.ntile, p.rows);
  KDA_NORM_SHAPES(Wide<T>::E, KDA_NORM)
#undef KDA_NORM
  return hipGetLastError();
}

// Rows per workgroup for the backward pass.  The plan must not depend on the addresses (the caller sizes
// the workspace before it has them), so it goes by the aligned shape; any shape can run under it.
static NormPlan norm_bwd_plan(int B, int H, int T, int D, int Ew) {
  const NormShape n = norm_shape(D, Ew, true);
  return norm_plan(B, H, T, n.NV ? kNormThreads / n.L : 1);
}

size_t norm_bwd_workspace_bytes(int B, int H, int T, int D, bool bf16) {
  if (T < 1) return 0;
  const NormPlan p = norm_bwd_plan(B, H, T, D, bf16 ? 8 : 4);
  return (size_t)B * H * p.ntile * 2 * D * sizeof(float);
}

template <typename T, bool PK>
static hipError_t norm_bwd(const void* x, const uint8_t* xs, const float* w, const float* mean, const float* rstd,
                           const void* dy, void* dx, float* part, int B, int H, int T_, int D, hipStream_t s) {
  const int grp = D < 32 ? D : 32;
  const NormPlan p = norm_bwd_plan(B, H, T_, D, Wide<T>::E);
  const dim3 grid((unsigned)(B * H * p.ntile));
  const T* xt = PK ? nullptr : (const T*)x;
  const uint8_t* xc = PK ? (const uint8_t*)x : nullptr;
  const NormShape n = norm_shape(D, Wide<T>::E, aligned16(x, dy, dx));
  if (n.NV == 0) {
    hipLaunchKernelGGL((norm_bwd_any_kernel<T, PK>), grid, dim3(kNormThreads), 0, s, xt, xc, xs, w, mean, rstd,
                       (const T*)dy, (T*)dx, part, H, T_, D, grp, p.ntile, p.rows);
    return hipGetLastError();
  }
#define KDA_NORM(E_, L_, NV_)                                                                                         \
  if (n.E == E_ && n.L == L_ && n.NV == NV_)                                                                          \
    hipLaunchKernelGGL((norm_bwd_kernel<T, E_, L_, NV_, PK>), grid, dim3(kNormThreads), 0, s, xt, xc, xs, w, mean,    \
                       rstd, (const T*)dy, (T*)dx, part, H, T_, D, grp, p.ntile, p.rows);
  KDA_NORM_SHAPES(Wide<T>::E, KDA_NORM)
#undef KDA_NORM
  return hipGetLastError();
}

template <typename T>
hipError_t launch_norm_bwd(const void* x, const uint8_t* x_scales, const float* w, const float* mean,
                           const float* rstd, const void* dy, void* dx, float* dw, float* db, void* workspace, int B,
                           int H, int T_, int D, hipStream_t s) {
  float* part = (dw || db) ? reinterpret_cast<float*>(workspace) : nullptr;
  int ntile = 0;
  if (T_ > 0) {
    ntile = norm_bwd_plan(B, H, T_, D, Wide<T>::E).ntile;
    const hipError_t e = x_scales ? norm_bwd<T, true>(x, x_scales, w, mean, rstd, dy, dx, part, B, H, T_, D, s)
                                  : norm_bwd<T, false>(x, x_scales, w, mean, rstd, dy, dx, part, B, H, T_, D, s);
    if (e != hipSuccess) return e;
  }
  if (dw || db) {                                  // (T = 0: both come out zero)
    const int ncol = (2 * D + 63) / 64;
    hipLaunchKernelGGL(norm_bwd_reduce_kernel, dim3((unsigned)(H * ncol)), dim3(256), 0, s, part, dw, db, B, H, D,
                       ntile, ncol);
  }
  return hipGetLastError();
}

#define KDA_INST(T)                                                                                                   \
  template hipError_t launch_norm_fwd<T>(const void*, const float*, const float*, float, void*, float*, float*, int, \
                                         int, int, int, hipStream_t);                                                 \
  template hipError_t launch_norm_bwd<T>(const void*, const uint8_t*, const float*, const float*, const float*,       \
                                         const void*, void*, float*, float*, void*, int, int, int, int, hipStream_t);
KDA_INST(float)
KDA_INST(bf16_t)
#undef KDA_INST

}  // namespace kda
