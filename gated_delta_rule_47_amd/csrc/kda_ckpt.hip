// Activations in 8 bits for the backward pass: OCP e4m3 codes with one power-of-two scale per group of
// G = min(D, 32) channels of a row, kept as the byte e + 127.  e is the smallest exponent >= -127 with
// amax <= 448 * 2^e over the group's finite values, so nothing saturates; scaling by 2^-e is exact and
// the one rounding is that to e4m3 (nearest even).  Infinities and NaN become NaN (e4m3 has no
// infinity) and do not move their group's scale.  Bound by memory: one read, one write; 8 channels per thread
// (16 bytes of bf16, 8 of codes), a group's maximum taken among its lanes.  2 x 32 x 8192 rows of 128, bf16: pack
// 39 us (5.3 TB/s), unpack 30 us (6.8 TB/s, two thirds of it writes); fp32, both 154 us (4.4 TB/s).
#include "kda_decay_attn.h"
#include "kda_launch.h"

namespace kda {

constexpr uint32_t kExpMask = 0x7f800000u;

__device__ __forceinline__ bool finite_bits(uint32_t u) { return (u & kExpMask) != kExpMask; }

// The exponent e for the largest finite magnitude of a group, given as its bits.  With amax = m 2^p,
// m in [1, 2): 448 = 1.75 * 2^8, so e = p - 8, or p - 7 if m > 1.75.
__device__ __forceinline__ int group_exp(uint32_t amax) {
  const int p = (int)(amax >> 23) - 127;         // (a subnormal's p comes out -127: clamped below anyway)
  const int e = p - 8 + ((amax & 0x7fffffu) > 0x600000u ? 1 : 0);
  return e < -127 ? -127 : e;
}
__device__ __forceinline__ float exp2_int(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }  // -126..127

// x * 2^-e (exact up to values that round to zero in e4m3), not finite -> NaN
__device__ __forceinline__ float scaled_down(float x, int e) {
  return finite_bits(__float_as_uint(x)) ? x * exp2_int(-e) : __uint_as_float(0x7fc00000u);
}
__device__ __forceinline__ uint32_t code4(const float* f) {
  int u = __builtin_amdgcn_cvt_pk_fp8_f32(f[0], f[1], 0, false);
  u = __builtin_amdgcn_cvt_pk_fp8_f32(f[2], f[3], u, true);
  return (uint32_t)u;
}

template <typename T> __device__ __forceinline__ void get8(const T* p, float* f);
template <> __device__ __forceinline__ void get8<bf16_t>(const bf16_t* p, float* f) {
  const u32x4_t u = *reinterpret_cast<const u32x4_t*>(p);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(u[i] << 16);
    f[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
  }
}
template <> __device__ __forceinline__ void get8<float>(const float* p, float* f) {
  const floatx4 a = *reinterpret_cast<const floatx4*>(p), b = *reinterpret_cast<const floatx4*>(p + 4);
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = a[i], f[4 + i] = b[i];
}
template <typename T> __device__ __forceinline__ void put8(T* p, const float* f);
template <> __device__ __forceinline__ void put8<bf16_t>(bf16_t* p, const float* f) {
  *reinterpret_cast<u32x4_t*>(p) = u32x4_t{pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                                           pack_bf16x2(f[6], f[7])};
}
template <> __device__ __forceinline__ void put8<float>(float* p, const float* f) {
  *reinterpret_cast<floatx4*>(p) = floatx4{f[0], f[1], f[2], f[3]};
  *reinterpret_cast<floatx4*>(p + 4) = floatx4{f[4], f[5], f[6], f[7]};
}

// Eight channels per thread; LG = G / 8 lanes (1, 2 or 4) share a group.  The tensor is one run of
// n8 such pieces, since a row is a whole number of groups.
template <typename T, int LG>
__global__ void __launch_bounds__(256) ckpt_pack_kernel(const T* __restrict__ x, uint8_t* __restrict__ codes,
                                                        uint8_t* __restrict__ scales, long long n8) {
  const long long step = (long long)gridDim.x * 256;
  for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i - threadIdx.x % LG < n8; i += step) {
    // (a group's lanes leave the loop together: n8 is a multiple of LG)
    float f[8];
    get8<T>(x + 8 * i, f);
    uint32_t m = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint32_t u = __float_as_uint(f[e]) & 0x7fffffffu;
      m = max(m, finite_bits(u) ? u : 0u);
    }
#pragma unroll
    for (int d = 1; d < LG; d <<= 1) m = max(m, (uint32_t)__shfl_xor((int)m, d, 64));
    const int e = group_exp(m);
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = scaled_down(f[j], e);
    *reinterpret_cast<u32x2_t*>(codes + 8 * i) = u32x2_t{code4(f), code4(f + 4)};
    if (threadIdx.x % LG == 0) scales[i / LG] = (uint8_t)(e + 127);
  }
}

// Any D <= 32 or multiple of 32, any alignment: one thread per group.
template <typename T>
__global__ void __launch_bounds__(256) ckpt_pack_any_kernel(const T* __restrict__ x, uint8_t* __restrict__ codes,
                                                            uint8_t* __restrict__ scales, long long ngroup, int G) {
  const long long step = (long long)gridDim.x * 256;
  for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < ngroup; i += step) {
    uint32_t m = 0;
    for (int j = 0; j < G; ++j) {
      const uint32_t u = __float_as_uint(to_f<T>(x[i * G + j])) & 0x7fffffffu;
      m = max(m, finite_bits(u) ? u : 0u);
    }
    const int e = group_exp(m);
    for (int j = 0; j < G; ++j)
      codes[i * G + j] = (uint8_t)__builtin_amdgcn_cvt_pk_fp8_f32(scaled_down(to_f<T>(x[i * G + j]), e), 0.0f, 0, false);
    scales[i] = (uint8_t)(e + 127);
  }
}

template <typename T, int LG>
__global__ void __launch_bounds__(256) ckpt_unpack_kernel(const uint8_t* __restrict__ codes,
                                                          const uint8_t* __restrict__ scales, T* __restrict__ x,
                                                          long long n8) {
  const long long step = (long long)gridDim.x * 256;
  for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < n8; i += step) {
    const u32x2_t u = *reinterpret_cast<const u32x2_t*>(codes + 8 * i);
    const float s = ckpt_scale(scales[i / LG]);
    float f[8];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const floatx2 a = __builtin_amdgcn_cvt_pk_f32_fp8((int)u[j], false);
      const floatx2 b = __builtin_amdgcn_cvt_pk_f32_fp8((int)u[j], true);
      f[4 * j] = a[0] * s;
      f[4 * j + 1] = a[1] * s;
      f[4 * j + 2] = b[0] * s;
      f[4 * j + 3] = b[1] * s;
    }
    put8<T>(x + 8 * i, f);
  }
}

template <typename T>
__global__ void __launch_bounds__(256) ckpt_unpack_any_kernel(const uint8_t* __restrict__ codes,
                                                              const uint8_t* __restrict__ scales, T* __restrict__ x,
                                                              long long n, int G) {
  const long long step = (long long)gridDim.x * 256;
  for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < n; i += step) {
    const floatx2 a = __builtin_amdgcn_cvt_pk_f32_fp8((int)codes[i], false);
    x[i] = from_f<T>(a[0] * ckpt_scale(scales[i / G]));
  }
}

// ------------------------------------------------------------------ launchers
static unsigned ckpt_grid(long long threads) {
  const long long b = (threads + 255) / 256;
  return (unsigned)(b < 16384 ? b : 16384);
}
static bool ckpt_wide(const void* x, const void* codes, int G) {
  return (G == 8 || G == 16 || G == 32) && ((uintptr_t)x & 15) == 0 && ((uintptr_t)codes & 7) == 0;
}

template <typename T>
hipError_t launch_ckpt_pack(const void* x, uint8_t* codes, uint8_t* scales, long long rows, int D, hipStream_t s) {
  const int G = D < 32 ? D : 32;
  const long long n = rows * D;
  if (n == 0) return hipSuccess;
  if (!ckpt_wide(x, codes, G)) {
    hipLaunchKernelGGL(ckpt_pack_any_kernel<T>, dim3(ckpt_grid(n / G)), dim3(256), 0, s, (const T*)x, codes, scales,
                       n / G, G);
  } else {
    const dim3 grid(ckpt_grid(n / 8));
    if (G == 32)
      hipLaunchKernelGGL((ckpt_pack_kernel<T, 4>), grid, dim3(256), 0, s, (const T*)x, codes, scales, n / 8);
    else if (G == 16)
      hipLaunchKernelGGL((ckpt_pack_kernel<T, 2>), grid, dim3(256), 0, s, (const T*)x, codes, scales, n / 8);
    else
      hipLaunchKernelGGL((ckpt_pack_kernel<T, 1>), grid, dim3(256), 0, s, (const T*)x, codes, scales, n / 8);
  }
  return hipGetLastError();
}

template <typename T>
hipError_t launch_ckpt_unpack(const uint8_t* codes, const uint8_t* scales, void* x, long long rows, int D,
                              hipStream_t s) {
  const int G = D < 32 ? D : 32;
  const long long n = rows * D;
  if (n == 0) return hipSuccess;
  if (!ckpt_wide(x, codes, G)) {
    hipLaunchKernelGGL(ckpt_unpack_any_kernel<T>, dim3(ckpt_grid(n)), dim3(256), 0, s, codes, scales, (T*)x, n, G);
  } else {
    const dim3 grid(ckpt_grid(n / 8));
    if (G == 32)
      hipLaunchKernelGGL((ckpt_unpack_kernel<T, 4>), grid, dim3(256), 0, s, codes, scales, (T*)x, n / 8);
    else if (G == 16)
      hipLaunchKernelGGL((ckpt_unpack_kernel<T, 2>), grid, dim3(256), 0, s, codes, scales, (T*)x, n / 8);
    else
      hipLaunchKernelGGL((ckpt_unpack_kernel<T, 1>), grid, dim3(256), 0, s, codes, scales, (T*)x, n / 8);
  }
  return hipGetLastError();
}

template hipError_t launch_ckpt_pack<float>(const void*, uint8_t*, uint8_t*, long long, int, hipStream_t);
template hipError_t launch_ckpt_pack<bf16_t>(const void*, uint8_t*, uint8_t*, long long, int, hipStream_t);
template hipError_t launch_ckpt_unpack<float>(const uint8_t*, const uint8_t*, void*, long long, int, hipStream_t);
template hipError_t launch_ckpt_unpack<bf16_t>(const uint8_t*, const uint8_t*, void*, long long, int, hipStream_t);

}  // namespace kda
