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
// bf16: forward, 32768 rows of 512, 13 us (5.2 TB/s); backward, 2 x 32 heads of 8192 rows of 128, 85 us with the
// reduction's 4 (4.8 TB/s), from 8-bit x 69 (4.9 TB/s); 4096 rows of 16384, forward 51 (5.3), backward 121 (3.3, 20 of
// them the reduction).  fp32: forward, 32768 rows of 512, 25 (5.4); backward, the heads above, 162 (5.0), from 8 bits 124.
#include <type_traits>

#include "kda_decay_attn.h"
#include "kda_launch.h"

namespace kda {

constexpr int kNormThreads = 256;

// Sum over the L lanes of a row: a power of two up to 64, or the whole workgroup (whose four waves add
// in a fixed order through `red`); every lane of the row gets it.
// Lanes exchange within the register file (DPP within 16 lanes, lane swaps beyond), not through LDS.
template <int CTRL> __device__ __forceinline__ float dpp(float x) {
  return __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(x), CTRL, 0xf, 0xf, true));
}
template <int L> __device__ __forceinline__ float row_sum(float x, float* red) {
  if constexpr (L >= 2) x += dpp<0xB1>(x);       // lane ^ 1
  if constexpr (L >= 4) x += dpp<0x4E>(x);       // lane ^ 2
  if constexpr (L >= 8) x += dpp<0x141>(x);      // mirrored in 8: the other four's sum
  if constexpr (L >= 16) x += dpp<0x140>(x);     // mirrored in 16: the other eight's
  if constexpr (L >= 32) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    x = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  }
  if constexpr (L >= 64) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    x = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  }
  if constexpr (L > 64) {
    static_assert(L == kNormThreads, "rows of a wave or of the workgroup");
    __syncthreads();
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = x;
    __syncthreads();
    x = (red[0] + red[1]) + (red[2] + red[3]);
  }
  return x;
}

// E consecutive elements of a row, 16 bytes: rows may start at any element, and global memory takes a
// 16-byte access at any address.  n < E: the last vector of a row, whose elements are taken one by one.
template <typename T> struct Wide {
  static constexpr int E = 16 / (int)sizeof(T);
};
template <int N, int A> struct __attribute__((packed, aligned(A))) Words {
  uint32_t u[N];
};
template <typename T> struct Raw {                // as loaded
  static constexpr int E = Wide<T>::E;
  uint32_t u[4];
  __device__ __forceinline__ void load(const T* p, int n) {
    if (n == E) {
      const Words<4, sizeof(T)> x = *reinterpret_cast<const Words<4, sizeof(T)>*>(p);
#pragma unroll
      for (int i = 0; i < 4; ++i) u[i] = x.u[i];
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (E == 4) {
          u[i] = i < n ? __float_as_uint(p[i]) : 0u;
        } else {
          const uint32_t lo = 2 * i < n ? p[2 * i] : 0u, hi = 2 * i + 1 < n ? p[2 * i + 1] : 0u;
          u[i] = hi << 16 | lo;
        }
      }
    }
  }
  __device__ __forceinline__ void get(float* f) const {
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
};
// E entries of a head's parameter row (n of them in the row), or the same value for a row that is not there
template <int E> __device__ __forceinline__ void params(const float* p, int n, float none, float* f) {
  if (p && n == E) {
    const Words<E, 4> x = *reinterpret_cast<const Words<E, 4>*>(p);
#pragma unroll
    for (int e = 0; e < E; ++e) f[e] = __uint_as_float(x.u[e]);
  } else {
#pragma unroll
    for (int e = 0; e < E; ++e) f[e] = p && e < n ? p[e] : none;
  }
}
template <typename T> __device__ __forceinline__ void vec_put(T* p, const float* f, int n) {
  constexpr int E = Wide<T>::E;
  if (n == E) {
    Words<4, sizeof(T)> x;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (E == 4) x.u[i] = __float_as_uint(f[i]);
      else x.u[i] = pack_bf16x2(f[2 * i], f[2 * i + 1]);
    }
    *reinterpret_cast<Words<4, sizeof(T)>*>(p) = x;
  } else {
#pragma unroll
    for (int e = 0; e < E; ++e)
      if (e < n) p[e] = from_f<T>(f[e]);
  }
}
template <typename T> struct RawCodes {           // E codes of an 8-bit tensor and their scale byte
  static constexpr int E = Wide<T>::E;
  uint32_t u[E / 4], sc;
  __device__ __forceinline__ void load(const uint8_t* p, const uint8_t* s, int n) {
    sc = *s;
    if (n == E) {
      const Words<E / 4, 1> x = *reinterpret_cast<const Words<E / 4, 1>*>(p);
#pragma unroll
      for (int i = 0; i < E / 4; ++i) u[i] = x.u[i];
    } else {
#pragma unroll
      for (int i = 0; i < E / 4; ++i) {
        u[i] = 0;
#pragma unroll
        for (int b = 0; b < 4; ++b)
          if (4 * i + b < n) u[i] |= (uint32_t)p[4 * i + b] << 8 * b;
      }
    }
  }
  __device__ __forceinline__ void get(float* f) const {
    const float s = ckpt_scale(sc);
#pragma unroll
    for (int i = 0; i < E / 4; ++i) {
      const floatx2 a = __builtin_amdgcn_cvt_pk_f32_fp8((int)u[i], false);
      const floatx2 b = __builtin_amdgcn_cvt_pk_f32_fp8((int)u[i], true);
      f[4 * i] = a[0] * s;
      f[4 * i + 1] = a[1] * s;
      f[4 * i + 2] = b[0] * s;
      f[4 * i + 3] = b[1] * s;
    }
  }
};

// Value i of an 8-bit tensor with D channels, one scale byte per `grp` channels.
__device__ __forceinline__ float ckpt_value(const uint8_t* codes, const uint8_t* sc, size_t row, int i, int D,
                                            int grp) {
  const floatx2 a = __builtin_amdgcn_cvt_pk_f32_fp8((int)codes[row * D + i], false);
  return a[0] * ckpt_scale(sc[row * (D / grp) + i / grp]);
}

// (var + eps)^-1/2; a variance that rounding left below zero is zero, NaN stays NaN
__device__ __forceinline__ float rstd_of(float var, float eps) { return 1.0f / sqrtf((var < 0.0f ? 0.0f : var) + eps); }

// Rows of one of the tiles of tile_rows rows that a head's T rows are cut into (the last may be short).  The kernels
// count rows from the tile's first one: T may be next to 2^31, where the end of the last tile, or a row a step
// behind the last one, is past an int.
__device__ __forceinline__ int rows_of_tile(int T, int tile, int tile_rows) {
  return min(tile_rows, T - tile * tile_rows);
}

// ------------------------------------------------------------------ forward
// TAIL: D is not a multiple of E, so a row's last vector holds fewer elements.
template <typename T, int L, int NV, bool TAIL>
__global__ void __launch_bounds__(kNormThreads) norm_fwd_kernel(const T* __restrict__ x, const float* __restrict__ w,
                                                                const float* __restrict__ b, float eps,
                                                                T* __restrict__ y, float* __restrict__ mean,
                                                                float* __restrict__ rstd, int H, int T_, int D,
                                                                int ntile, int tile_rows) {
  constexpr int E = Wide<T>::E, RPW = kNormThreads / L;
  __shared__ float rsum[kNormThreads / 64];
  const int bh = blockIdx.x / ntile, tile = blockIdx.x - bh * ntile;
  const int c = threadIdx.x % L, rr = threadIdx.x / L;
  const float inv = 1.0f / (float)D;
  float wv[NV][E], bv[NV][E];
  int n[NV];                                       // elements of this lane's vectors
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int col = (c + i * L) * E;
    n[i] = min(max(D - col, 0), E);
    const size_t at = (size_t)(bh % H) * D + col;
    params<E>(w ? w + at : nullptr, n[i], 1.0f, wv[i]);
    params<E>(b ? b + at : nullptr, n[i], 0.0f, bv[i]);
  }
  const auto has = [&](int i, int e) { return TAIL ? e < n[i] : n[i] > 0; };
  const int nrow = rows_of_tile(T_, tile, tile_rows);
  const size_t row0 = (size_t)bh * T_ + (size_t)tile * tile_rows;
  Raw<T> next[NV];                                 // the row after this one, requested before this one's sums
  const auto request = [&](int t) {
    if (t < nrow) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (n[i] > 0) next[i].load(x + (row0 + t) * D + (c + i * L) * E, TAIL ? n[i] : E);
    }
  };
  request(rr);
  for (int t = rr; t < nrow; t += RPW) {
    const size_t row = row0 + t;
    float v[NV][E];
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      next[i].get(v[i]);
#pragma unroll
      for (int e = 0; e < E; ++e) s += has(i, e) ? v[i][e] : 0.0f;
    }
    request(t + RPW);
    const float m = row_sum<L>(s, rsum) * inv;
    float q = 0.0f, d = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < E; ++e) {
        v[i][e] = has(i, e) ? v[i][e] - m : 0.0f;
        q = fmaf(v[i][e], v[i][e], q);
        d += v[i][e];
      }
    // m is rounded (by up to 2^-24 |m|, which shows where a row's mean is far above its spread): what is
    // left of the mean in the differences is taken out of them and of their squares
    const float dm = row_sum<L>(d, rsum) * inv;
    const float r = rstd_of(row_sum<L>(q, rsum) * inv - dm * dm, eps);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
#pragma unroll
      for (int e = 0; e < E; ++e) v[i][e] = fmaf((v[i][e] - dm) * r, wv[i][e], bv[i][e]);
      if (n[i] > 0) vec_put<T>(y + row * D + (c + i * L) * E, v[i], TAIL ? n[i] : E);
    }
    if (c == 0) {
      if (mean) mean[row] = m + dm;
      if (rstd) rstd[row] = r;
    }
  }
}

// Any width: a workgroup per row, which is read three times (the second and third time
// from cache for rows that fit it), an element per lane.  fp32, 4096 rows of 12288: 160 us, 2.5 TB/s.
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
template <typename T, int L, int NV, bool TAIL, bool PK>
__global__ void __launch_bounds__(kNormThreads)
    norm_bwd_kernel(const T* __restrict__ x, const uint8_t* __restrict__ xc, const uint8_t* __restrict__ xs,
                    const float* __restrict__ w, const float* __restrict__ mean, const float* __restrict__ rstd,
                    const T* dy, T* dx, float* __restrict__ part, int H, int T_, int D, int grp, int ntile,
                    int tile_rows) {
  constexpr int E = Wide<T>::E, RPW = kNormThreads / L;
  __shared__ float rsum[kNormThreads / 64];
  const int bh = blockIdx.x / ntile, tile = blockIdx.x - bh * ntile;
  const int c = threadIdx.x % L, rr = threadIdx.x / L;
  const float inv = 1.0f / (float)D;
  float wv[NV][E], dw[NV][E], db[NV][E];
  int n[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int col = (c + i * L) * E;
    n[i] = min(max(D - col, 0), E);
    params<E>(w ? w + (size_t)(bh % H) * D + col : nullptr, n[i], 1.0f, wv[i]);
#pragma unroll
    for (int e = 0; e < E; ++e) dw[i][e] = db[i][e] = 0.0f;
  }
  const int nrow = rows_of_tile(T_, tile, tile_rows);
  const size_t row0 = (size_t)bh * T_ + (size_t)tile * tile_rows;
  typename std::conditional<PK, RawCodes<T>, Raw<T>>::type nx[NV];
  Raw<T> ndy[NV];
  float nm = 0.0f, nr = 0.0f;
  const auto request = [&](int t) {
    if (t < nrow) {
      const size_t row = row0 + t;
      nm = mean[row];
      nr = rstd[row];
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (n[i] > 0) {
          const int col = (c + i * L) * E, k = TAIL ? n[i] : E;
          ndy[i].load(dy + row * D + col, k);
          if constexpr (PK) nx[i].load(xc + row * D + col, xs + row * (D / grp) + col / grp, k);
          else nx[i].load(x + row * D + col, k);
        }
    }
  };
  request(rr);
  for (int t = rr; t < nrow; t += RPW) {
    const size_t row = row0 + t;
    const float m = nm, r = nr;
    float xh[NV][E], g[NV][E];
    float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      ndy[i].get(g[i]);
      nx[i].get(xh[i]);
    }
    request(t + RPW);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (n[i] > 0) {
#pragma unroll
        for (int e = 0; e < E; ++e) {
          // (elements behind the row's end: dy = 0 there, and 0 in place of x's)
          xh[i][e] = !TAIL || e < n[i] ? (xh[i][e] - m) * r : 0.0f;
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
      if (n[i] > 0) {
#pragma unroll
        for (int e = 0; e < E; ++e) g[i][e] = r * (g[i][e] - c1 - xh[i][e] * c2);
        vec_put<T>(dx + row * D + (c + i * L) * E, g[i], TAIL ? n[i] : E);
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

// Any width: a workgroup takes the tile's rows one after another; a thread's columns
// (threadIdx.x + 256 i) keep their running sums in the workgroup's part of `part`.  dx may be dy, of which a thread
// reads an element for the last time before it writes it.  fp32, 4096 rows of 12288: 724 us with the reduction's 17,
// 0.83 TB/s: every row's terms of the sums go to memory and back.
template <typename T, bool PK>
__global__ void __launch_bounds__(kNormThreads)
    norm_bwd_any_kernel(const T* __restrict__ x, const uint8_t* __restrict__ xc, const uint8_t* __restrict__ xs,
                        const float* __restrict__ w, const float* __restrict__ mean, const float* __restrict__ rstd,
                        const T* dy, T* dx, float* part, int H, int T_, int D, int grp,
                        int ntile, int tile_rows) {
  __shared__ float red[kNormThreads / 64];
  const int bh = blockIdx.x / ntile, tile = blockIdx.x - bh * ntile;
  const float* wr = w ? w + (size_t)(bh % H) * D : nullptr;
  float* out = part ? part + (size_t)blockIdx.x * 2 * D : nullptr;
  const int nrow = rows_of_tile(T_, tile, tile_rows);
  const size_t row0 = (size_t)bh * T_ + (size_t)tile * tile_rows;
  for (int t = 0; t < nrow; ++t) {
    const size_t row = row0 + t;
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
        out[i] = (t == 0 ? 0.0f : out[i]) + d * xh;
        out[D + i] = (t == 0 ? 0.0f : out[D + i]) + d;
      }
    }
    const float c1 = row_sum<kNormThreads>(s1, red) / (float)D, c2 = row_sum<kNormThreads>(s2, red) / (float)D;
    for (int i = threadIdx.x; i < D; i += kNormThreads) {
      const float p = to_f<T>(dy[row * D + i]) * (wr ? wr[i] : 1.0f);
      dx[row * D + i] = from_f<T>(r * (p - c1 - xhat(i) * c2));
    }
  }
}

// Sums of the parts of a head's workgroups (2 D columns each: dw's, then db's), kRedParts of them into one
// at a time until one is left: part p of head h is row (p / nt * H + h) * nt + p % nt.  64 columns per
// workgroup, four threads per column over interleaved parts.
constexpr int kRedParts = 64;
__global__ void __launch_bounds__(256) norm_bwd_reduce_kernel(const float* __restrict__ part, int np, int nt,
                                                              float* __restrict__ out, float* __restrict__ dw,
                                                              float* __restrict__ db, int H, int D, int ncol,
                                                              int nout) {
  __shared__ float red[4][64];
  const int cb = blockIdx.x % ncol, hp = blockIdx.x / ncol, h = hp % H, po = hp / H;
  const int c = cb * 64 + (threadIdx.x & 63), sl = threadIdx.x >> 6;
  const int p0 = po * kRedParts, p1 = min(np, p0 + kRedParts);
  float s = 0.0f;
  if (c < 2 * D) {
#pragma unroll 8
    for (int p = p0 + sl; p < p1; p += 4) s += part[((size_t)(p / nt * H + h) * nt + p % nt) * 2 * D + c];
  }
  red[sl][threadIdx.x & 63] = s;
  __syncthreads();
  if (sl == 0 && c < 2 * D) {
    s = (red[0][threadIdx.x] + red[1][threadIdx.x]) + (red[2][threadIdx.x] + red[3][threadIdx.x]);
    if (nout > 1) out[((size_t)h * nout + po) * 2 * D + c] = s;
    else if (c < D) {
      if (dw) dw[(size_t)h * D + c] = s;
    } else if (db) {
      db[(size_t)h * D + c - D] = s;
    }
  }
}

// ------------------------------------------------------------------ launchers
// Rows of one workgroup: 32 where that leaves 512 workgroups (the weights are read, and partial sums
// written, once per workgroup), and no more than 1024 workgroups.  32768 rows of 512 bf16 in 512, 1024 and 2048 of
// them: forward 16.6, 13.6, 13.0 us, backward 24.1, 24.6, 25.4; 8192 rows of 4096 the same in all (26, 44).
struct NormPlan {
  int ntile, rows;
};
static NormPlan norm_plan(int B, int H, int T, int rpw) {
  const long long bh = (long long)B * H, total = bh * T;
  long long want = total / 32;
  if (want < 512) want = 512;
  if (want > 1024) want = 1024;
  long long tiles = (want + bh - 1) / bh;
  const long long most = ((long long)T + rpw - 1) / rpw;   // a step of the workgroup's rows at least
  if (tiles > most) tiles = most;
  if (tiles < 1) tiles = 1;
  long long rows = (T + tiles - 1) / tiles;
  rows = (rows + rpw - 1) / rpw * rpw;
  if (rows < 1) rows = 1;
  return NormPlan{(int)((T + rows - 1) / rows), (int)rows};
}

// How a row of D elements is held: L lanes, NV vectors of E elements per lane; the workgroup shares a row
// once one wave would need more than 32 fp32 registers for it.  NV = 0: wider than 8 vectors for each of
// 256 lanes, the any-width kernels run.
struct NormShape {
  int L, NV;
};
static NormShape norm_shape(int D, int E) {
  const int n = (D + E - 1) / E, wave_nv = 32 / E;
  NormShape p{1, 1};
  while (p.L < n && p.L < 64) p.L <<= 1;
  while (p.NV * p.L < n) p.NV <<= 1;
  if (p.NV > wave_nv) {
    p.L = kNormThreads;
    p.NV = wave_nv / 2;
    while (p.NV * p.L < n) p.NV <<= 1;
    if (p.NV > 8) p.NV = 0;
  }
  return p;
}
static int norm_rpw(const NormShape& n) { return n.NV ? kNormThreads / n.L : 1; }
// The shapes above as instances: CASE(L, NV), for those of them that rows of a type come to (norm_used).  Rows of
// 8-bit codes end inside a vector only up to 32 channels (wider ones are multiples of 32).
#define KDA_NORM_SHAPES(CASE)                                                                          \
  CASE(1, 1) CASE(2, 1) CASE(4, 1) CASE(8, 1) CASE(16, 1) CASE(32, 1) CASE(64, 1) CASE(64, 2)          \
  CASE(64, 4) CASE(64, 8) CASE(256, 2) CASE(256, 4) CASE(256, 8)
constexpr bool norm_used(int L, int NV, int E) { return L == kNormThreads ? NV >= 16 / E : NV <= 32 / E; }
constexpr bool norm_used(int L, int NV, int E, bool tail, bool packed) {
  return norm_used(L, NV, E) && !(tail && packed && L * E > 32);
}

template <typename T>
hipError_t launch_norm_fwd(const void* x, const float* w, const float* b, float eps, void* y, float* mean, float* rstd,
                           int B, int H, int T_, int D, hipStream_t s) {
  if (T_ == 0) return hipSuccess;
  const NormShape n = norm_shape(D, Wide<T>::E);
  if (n.NV == 0) {
    hipLaunchKernelGGL(norm_fwd_any_kernel<T>, dim3((unsigned)((size_t)B * H * T_)), dim3(kNormThreads), 0, s,
                       (const T*)x, w, b, eps, (T*)y, mean, rstd, H, T_, D);
    return hipGetLastError();
  }
  const NormPlan p = norm_plan(B, H, T_, norm_rpw(n));
  const dim3 grid((unsigned)(B * H * p.ntile));
  const bool tail = D % Wide<T>::E != 0;
#define KDA_NORM(L_, NV_)                                                                                             \
  if constexpr (norm_used(L_, NV_, Wide<T>::E)) {                                                                     \
    if (n.L == L_ && n.NV == NV_) {                                                                                   \
      if (tail)                                                                                                       \
        hipLaunchKernelGGL((norm_fwd_kernel<T, L_, NV_, true>), grid, dim3(kNormThreads), 0, s, (const T*)x, w, b,    \
                           eps, (T*)y, mean, rstd, H, T_, D, p.ntile, p.rows);                                        \
      else                                                                                                            \
        hipLaunchKernelGGL((norm_fwd_kernel<T, L_, NV_, false>), grid, dim3(kNormThreads), 0, s, (const T*)x, w, b,   \
                           eps, (T*)y, mean, rstd, H, T_, D, p.ntile, p.rows);                                        \
      return hipGetLastError();                                                                                       \
    }                                                                                                                 \
  }
  KDA_NORM_SHAPES(KDA_NORM)
#undef KDA_NORM
  return hipErrorInvalidValue;                     // (not reached)
}

// Partial sums of the workgroups, then those of the reduction's steps one behind the other.
size_t norm_bwd_workspace_bytes(int B, int H, int T, int D, bool bf16) {
  if (T < 1) return 0;
  const NormPlan p = norm_plan(B, H, T, norm_rpw(norm_shape(D, bf16 ? 8 : 4)));
  size_t rows = 0;
  for (long long np = (long long)B * p.ntile;; np = (np + kRedParts - 1) / kRedParts) {
    rows += (size_t)H * np;
    if (np <= kRedParts) break;
  }
  return rows * 2 * D * sizeof(float);
}

template <typename T, bool PK>
static hipError_t norm_bwd(const void* x, const uint8_t* xs, const float* w, const float* mean, const float* rstd,
                           const void* dy, void* dx, float* part, int B, int H, int T_, int D, const NormShape& n,
                           const NormPlan& p, hipStream_t s) {
  const int grp = D < 32 ? D : 32;
  const dim3 grid((unsigned)(B * H * p.ntile));
  const T* xt = PK ? nullptr : (const T*)x;
  const uint8_t* xc = PK ? (const uint8_t*)x : nullptr;
  const bool tail = D % Wide<T>::E != 0;
  if (n.NV == 0) {
    hipLaunchKernelGGL((norm_bwd_any_kernel<T, PK>), grid, dim3(kNormThreads), 0, s, xt, xc, xs, w, mean, rstd,
                       (const T*)dy, (T*)dx, part, H, T_, D, grp, p.ntile, p.rows);
    return hipGetLastError();
  }
#define KDA_NORM(L_, NV_)                                                                                              \
  if (n.L == L_ && n.NV == NV_) {                                                                                      \
    if constexpr (norm_used(L_, NV_, Wide<T>::E, true, PK)) {                                                          \
      if (tail) {                                                                                                      \
        hipLaunchKernelGGL((norm_bwd_kernel<T, L_, NV_, true, PK>), grid, dim3(kNormThreads), 0, s, xt, xc, xs, w,     \
                           mean, rstd, (const T*)dy, (T*)dx, part, H, T_, D, grp, p.ntile, p.rows);                    \
        return hipGetLastError();                                                                                      \
      }                                                                                                                \
    }                                                                                                                  \
    if constexpr (norm_used(L_, NV_, Wide<T>::E)) {                                                                    \
      if (!tail) {                                                                                                     \
        hipLaunchKernelGGL((norm_bwd_kernel<T, L_, NV_, false, PK>), grid, dim3(kNormThreads), 0, s, xt, xc, xs, w,    \
                           mean, rstd, (const T*)dy, (T*)dx, part, H, T_, D, grp, p.ntile, p.rows);                    \
        return hipGetLastError();                                                                                      \
      }                                                                                                                \
    }                                                                                                                  \
  }
  KDA_NORM_SHAPES(KDA_NORM)
#undef KDA_NORM
  return hipErrorInvalidValue;                     // (not reached)
}

template <typename T>
hipError_t launch_norm_bwd(const void* x, const uint8_t* x_scales, const float* w, const float* mean,
                           const float* rstd, const void* dy, void* dx, float* dw, float* db, void* workspace, int B,
                           int H, int T_, int D, hipStream_t s) {
  float* part = (dw || db) ? reinterpret_cast<float*>(workspace) : nullptr;
  const NormShape n = norm_shape(D, Wide<T>::E);
  const NormPlan p = norm_plan(B, H, T_, norm_rpw(n));
  if (T_ > 0) {
    const hipError_t e = x_scales ? norm_bwd<T, true>(x, x_scales, w, mean, rstd, dy, dx, part, B, H, T_, D, n, p, s)
                                  : norm_bwd<T, false>(x, x_scales, w, mean, rstd, dy, dx, part, B, H, T_, D, n, p, s);
    if (e != hipSuccess) return e;
  }
  if (dw || db) {                                  // (T = 0: no parts, both come out zero)
    const int ncol = (2 * D + 63) / 64;
    int np = T_ > 0 ? B * p.ntile : 0, nt = p.ntile > 0 ? p.ntile : 1;
    for (;;) {
      const int nout = np > kRedParts ? (np + kRedParts - 1) / kRedParts : 1;
      float* out = part ? part + (size_t)H * np * 2 * D : nullptr;
      hipLaunchKernelGGL(norm_bwd_reduce_kernel, dim3((unsigned)((long long)H * ncol * nout)), dim3(256), 0, s, part,
                         np, nt, out, dw, db, H, D, ncol, nout);
      if (nout == 1) break;
      part = out, np = nout, nt = nout;            // part p of head h at row h * nout + p from here on
    }
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
