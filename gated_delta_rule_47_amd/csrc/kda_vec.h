// Building blocks of the kernels that stream rows of channels: a few consecutive elements per lane, sums over a
// power of two of lanes, and the sum of workgroups' parts in a fixed order.
#pragma once

#include "kda_common.h"

namespace kda {

// A lane's N words at any address that holds an element: global memory takes a 16-byte access anywhere.
template <int N, int A> struct __attribute__((packed, aligned(A))) Words {
  uint32_t u[N];
};

// N consecutive elements of a row as loaded (N * sizeof(T) a multiple of 4), and as floats.
template <typename T, int N> struct Elems {
  static constexpr int M = N * (int)sizeof(T) / 4;
  uint32_t u[M];
  __device__ __forceinline__ void load(const T* p) {
    const Words<M, sizeof(T)> x = *reinterpret_cast<const Words<M, sizeof(T)>*>(p);
#pragma unroll
    for (int i = 0; i < M; ++i) u[i] = x.u[i];
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < M; ++i) u[i] = 0;
  }
  __device__ __forceinline__ float at(int i) const {
    if constexpr (sizeof(T) == 4) return __uint_as_float(u[i]);
    else return __uint_as_float((i & 1) ? u[i >> 1] & 0xffff0000u : u[i >> 1] << 16);
  }
  __device__ __forceinline__ void store(T* p) const {
    Words<M, sizeof(T)> x;
#pragma unroll
    for (int i = 0; i < M; ++i) x.u[i] = u[i];
    *reinterpret_cast<Words<M, sizeof(T)>*>(p) = x;
  }
  __device__ __forceinline__ void set(const float* f) {
#pragma unroll
    for (int i = 0; i < M; ++i) {
      if constexpr (sizeof(T) == 4) u[i] = __float_as_uint(f[i]);
      else u[i] = pack_bf16x2(f[2 * i], f[2 * i + 1]);
    }
  }
};

template <int N> __device__ __forceinline__ void load_f32(const float* p, float* f) {
  const Words<N, 4> x = *reinterpret_cast<const Words<N, 4>*>(p);
#pragma unroll
  for (int i = 0; i < N; ++i) f[i] = __uint_as_float(x.u[i]);
}

// Sum over L neighbouring lanes, L a power of two up to 64; every one of them gets it.
// Lanes exchange within the register file (DPP within 16 lanes, lane swaps beyond), not through LDS.
template <int CTRL> __device__ __forceinline__ float dpp(float x) {
  return __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(x), CTRL, 0xf, 0xf, true));
}
template <int L> __device__ __forceinline__ float lane_sum(float x) {
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
  return x;
}

// Sum over parts of float32 values: part p of value i stands at in[p * stride + i].  64 values per workgroup and 16
// lanes per value, each taking every 16th part in ascending order, then the 16 in a fixed order (repeatable bit by
// bit).  put(i, sum) stores value i.
constexpr int kSumThreads = 1024;
template <typename Put>
__device__ __forceinline__ void sum_parts(const float* in, size_t stride, int parts, int n, Put put) {
  __shared__ float red[16][64];
  const int lane = threadIdx.x & 63, row = threadIdx.x >> 6;
  const int i = blockIdx.x * 64 + lane;
  float s = 0.f;
  if (i < n) {
    const float* p = in + i;
#pragma unroll 8
    for (int k = row; k < parts; k += 16) s += p[(size_t)k * stride];
  }
  red[row][lane] = s;
  __syncthreads();
  if (row == 0 && i < n) {
    float t[16];
#pragma unroll
    for (int k = 0; k < 16; ++k) t[k] = red[k][lane];
#pragma unroll
    for (int w = 8; w; w >>= 1)
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (k < w) t[k] += t[k + w];
    put(i, t[0]);
  }
}

}  // namespace kda
