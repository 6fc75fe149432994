// Linear attention with a constant decay per head, S_t = a S_{t-1} + k_t v_t^T, o_t = S_t^T q_t
// with a = exp(log_decay[h]), evaluated in chunks of C tokens (gfx950).
//
// One kernel, the walk, serves the forward and all three gradients.  For operands Q, K, V and a
// state S (KD x VD) it computes, chunk by chunk (i, j token indices in a chunk of n tokens),
//   forward   O_i = r a^{i+1} Q_i^T S + c sum_{j<=i} a^{i-j} (Q_i.K_j) V_j,   S <- a^n S + u sum_j a^{n-1-j} K_j V_j^T
//   reverse   O_i = r a^{n-1-i} Q_i^T S + c sum_{j>=i} a^{j-i} (Q_i.K_j) V_j, S <- a^n S + u sum_j a^{j+1} K_j V_j^T
// (the reverse walk takes the chunks from last to first).  With R = dL/dS the gradients are
//   dq = forward(d_o, v, k; S^T), c = r = scale, u = 1
//   dk = reverse(v, d_o, q; R^T), dv = reverse(k, q, d_o; R), c = u = scale, r = 1; R at the start is d_state_in.
//
// A workgroup walks one segment of the tokens for one head and one tile of VT value columns with
// eight waves in two roles.  State waves hold S (KD x VT, fp32) in accumulators, a 2 x 2 split, and
// leave its bf16 (or fp32) image in LDS for the next chunk; output waves each own 16 tokens: their
// scores K Q^T come out of the matrix unit in the layout in which the product with V takes them, so
// the scores never touch LDS.  The roles overlap on every SIMD and meet at one barrier per chunk.
#pragma once

#include <type_traits>

#include "kda_common.h"

namespace kda {

// Operands of the walk; a tensor's `*_sc` are the scale bytes of its 8-bit form or null.
struct WalkArgs {
  const void *q, *k, *v;
  const uint8_t *q_sc, *k_sc, *v_sc;
  const float* log_decay;    // (H)
  const int* lengths;        // (B) or null
  const float* state_in;     // element (i, j) of head bh at bh * K * V + i * si_k + j * si_v; null = 0
  const float* seg_state;    // states at the segments' starts (B*H, nseg, K, V), same strides; used if nseg > 1
  float* state_out;          // the end state, null = not written (same strides)
  void* o;
  float c, r, u;             // scales of the intra-chunk term, the read and the update
  int si_k, si_v;
  int BH, H, T, K, V;        // K, V: the walk's key and value widths
  int nseg, seglen;          // seglen: a multiple of the chunk
  int zero_tail;             // write zeros to the rows of o behind a sequence's length
};

// Local states of the segments (all but the last in walking order), without the start state.
struct SegArgs {
  const void *k, *v;
  const uint8_t *k_sc, *v_sc;
  const float* log_decay;
  const int* lengths;
  float* seg_state;          // (B*H, nseg, K, V)
  float u;
  int BH, H, T, K, V, nseg, seglen;
};

typedef unsigned int u32x4_t __attribute__((ext_vector_type(4)));
typedef unsigned int u32x2_t __attribute__((ext_vector_type(2)));
typedef short short4v_t __attribute__((ext_vector_type(4)));

// ------------------------------------------------------------------ operand layouts
// A product's contraction runs in groups of DG indices.  A fragment holds, for row (or column)
// lane % 16 and lane group g = lane / 16, DG / 4 of the group's indices: DG / 4 consecutive ones
// when read along memory (`nat`), or those in which NACC accumulator tiles hold them (`from_acc`:
// index 16 n + 4 g + r of tile n).  `tr` reads the transpose of a [index][column] tile in the
// accumulator order.  Tile `ct` of 16 rows covers the rows row_of(ct, m), m = 0..15, which give a
// lane's accumulator registers of NACC adjacent tiles DG / 4 consecutive rows.
template <typename T> struct Lin;

template <> struct Lin<bf16_t> {                 // v_mfma_f32_16x16x32_bf16
  static constexpr int DG = 32, NACC = 2, EPP = 8, PAD = 8, SPLIT = 2;
  typedef short8 frag;
  static __device__ __forceinline__ int row_of(int ct, int m) {
    return 32 * (ct >> 1) + 8 * (m >> 2) + 4 * (ct & 1) + (m & 3);
  }
  static __device__ __forceinline__ frag nat(const bf16_t* row, int d0, int lane) {
    return *reinterpret_cast<const short8*>(row + d0 + 8 * (lane >> 4));
  }
  // two transposing reads: lane 4r + m of a group of 16 addresses row 4g + r (then 16 + 4g + r) at
  // four columns and lane j receives column j of the group's 16
  template <bool PERM> static __device__ __forceinline__ frag tr(const bf16_t* base, int ld, int ct, int d0, int lane) {
    const int g = lane >> 4, r = (lane >> 2) & 3, m = lane & 3;
    const int col = PERM ? 32 * (ct >> 1) + 8 * m + 4 * (ct & 1) : 16 * ct + 4 * m;
    const bf16_t* p = base + (d0 + 4 * g + r) * ld + col;
    const short4v_t a = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
        (__attribute__((address_space(3))) short4v_t*)(__attribute__((address_space(3))) const void*)p);
    const short4v_t b = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
        (__attribute__((address_space(3))) short4v_t*)(__attribute__((address_space(3))) const void*)(p + 16 * ld));
    return short8{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
  }
  static __device__ __forceinline__ floatx4 mma(frag a, frag b, floatx4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0,
                                                   0, 0);
  }
  static __device__ __forceinline__ frag from_acc(const floatx4* x) {
    return __builtin_bit_cast(short8, u32x4_t{pack_bf16x2(x[0][0], x[0][1]), pack_bf16x2(x[0][2], x[0][3]),
                                              pack_bf16x2(x[1][0], x[1][1]), pack_bf16x2(x[1][2], x[1][3])});
  }
  // x f as bf16 parts hi + lo, off by at most 2^-18 of the product: the state is returned in fp32, and
  // one bf16 rounding of the decayed operand (2^-9) would show in it
  static __device__ __forceinline__ void scaled(frag x, const float* f, frag* out) {
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float a = bf2f((bf16_t)x[2 * e]) * f[2 * e], b = bf2f((bf16_t)x[2 * e + 1]) * f[2 * e + 1];
      hi[e] = pack_bf16x2(a, b);
      lo[e] = pack_bf16x2(a - __uint_as_float(hi[e] << 16), b - __uint_as_float(hi[e] & 0xffff0000u));
    }
    out[0] = __builtin_bit_cast(short8, u32x4_t{hi[0], hi[1], hi[2], hi[3]});
    out[1] = __builtin_bit_cast(short8, u32x4_t{lo[0], lo[1], lo[2], lo[3]});
  }
  // token (within a group of DG) of fragment element e in the accumulator order
  static __device__ __forceinline__ int tok_of(int e, int g) { return 16 * (e >> 2) + 4 * g + (e & 3); }
  static __device__ __forceinline__ void store4(bf16_t* p, floatx4 x) {
    *reinterpret_cast<u32x2_t*>(p) = u32x2_t{pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3])};
  }
};

template <> struct Lin<float> {                  // four v_mfma_f32_16x16x4_f32
  static constexpr int DG = 16, NACC = 1, EPP = 4, PAD = 4, SPLIT = 1;
  typedef floatx4 frag;
  static __device__ __forceinline__ int row_of(int ct, int m) { return 16 * ct + m; }
  static __device__ __forceinline__ frag nat(const float* row, int d0, int lane) {
    return *reinterpret_cast<const floatx4*>(row + d0 + 4 * (lane >> 4));
  }
  template <bool PERM> static __device__ __forceinline__ frag tr(const float* base, int ld, int ct, int d0, int lane) {
    const float* p = base + (d0 + 4 * (lane >> 4)) * ld + 16 * ct + (lane & 15);
    return floatx4{p[0], p[ld], p[2 * ld], p[3 * ld]};
  }
  static __device__ __forceinline__ floatx4 mma(frag a, frag b, floatx4 c) {
#pragma unroll
    for (int r = 0; r < 4; ++r) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[r], b[r], c, 0, 0, 0);
    return c;
  }
  static __device__ __forceinline__ frag from_acc(const floatx4* x) { return x[0]; }
  static __device__ __forceinline__ void scaled(frag x, const float* f, frag* out) {
    out[0] = floatx4{x[0] * f[0], x[1] * f[1], x[2] * f[2], x[3] * f[3]};
  }
  static __device__ __forceinline__ int tok_of(int e, int g) { return 4 * g + e; }
  static __device__ __forceinline__ void store4(float* p, floatx4 x) { *reinterpret_cast<floatx4*>(p) = x; }
};

// ------------------------------------------------------------------ loads
// 2^(b - 127) for a scale byte b (b = 0: 2^-127, a subnormal).
__device__ __forceinline__ float ckpt_scale(uint32_t b) { return __uint_as_float(b ? b << 23 : 0x00400000u); }

// One piece of EPP consecutive channels of a row on its way from memory: 16 bytes of elements, or
// EPP codes and their group's scale byte.
template <typename T> struct Piece {
  u32x4_t raw;
  uint32_t sc;
  __device__ __forceinline__ u32x4_t elems(bool packed) const {
    if (!packed) return raw;
    const float s = ckpt_scale(sc);
    float f[8];
#pragma unroll
    for (int i = 0; i < Lin<T>::EPP / 4; ++i) {
      const floatx2 a = __builtin_amdgcn_cvt_pk_f32_fp8((int)raw[i], false);
      const floatx2 b = __builtin_amdgcn_cvt_pk_f32_fp8((int)raw[i], true);
      f[4 * i] = a[0] * s;
      f[4 * i + 1] = a[1] * s;
      f[4 * i + 2] = b[0] * s;
      f[4 * i + 3] = b[1] * s;
    }
    if constexpr (std::is_same<T, float>::value)
      return u32x4_t{__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3])};
    else
      return u32x4_t{pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                     pack_bf16x2(f[6], f[7])};
  }
};

// One head of a tensor (rows tokens x D channels) behind a range-checked buffer: rows from `len` on
// and channels from D on read as zero.
template <typename T, bool PK> struct HeadRows {
  __amdgpu_buffer_rsrc_t r, rs;
  int D, nsc;
  bool packed;
  __device__ __forceinline__ HeadRows(const void* base, const uint8_t* sc, int bh, int T_, int D_, int len) {
    D = D_;
    packed = PK && sc != nullptr;
    const int es = packed ? 1 : (int)sizeof(T);
    r = make_rsrc((const char*)base + (size_t)bh * T_ * D * es, (unsigned)len * (unsigned)(D * es));
    nsc = D < 32 ? 1 : D / 32;
    if (PK) rs = make_rsrc(sc + (packed ? (size_t)bh * T_ * nsc : 0), packed ? (unsigned)len * (unsigned)nsc : 0u);
  }
  __device__ __forceinline__ Piece<T> load(int t, int ch) const {
    Piece<T> p;
    const unsigned at = (unsigned)t * (unsigned)D + (unsigned)ch;
    const bool in = ch < D;
    if (PK && packed) {
      const unsigned off = in ? at : 0xfffffff0u;
      if constexpr (std::is_same<T, float>::value) {
        p.raw[0] = __builtin_amdgcn_raw_buffer_load_b32(r, off, 0, 0);
      } else {
        const u32x2_t x = __builtin_bit_cast(u32x2_t, __builtin_amdgcn_raw_buffer_load_b64(r, off, 0, 0));
        p.raw[0] = x[0];
        p.raw[1] = x[1];
      }
      p.sc = __builtin_amdgcn_raw_buffer_load_b8(rs, in ? (unsigned)t * (unsigned)nsc + (unsigned)(ch >> 5) : 0xfffffff0u,
                                                 0, 0);
    } else {
      p.raw = __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(
                                              r, in ? at * (unsigned)sizeof(T) : 0xfffffff0u, 0, 0));
    }
    return p;
  }
};

// A chunk of C rows x D channels (padded to DP) held by the NT threads between memory and LDS.
template <typename T, bool PK, int C, int DP, int NT> struct Stage {
  static constexpr int PPR = DP / Lin<T>::EPP, N = C * PPR, PER = (N + NT - 1) / NT;
  Piece<T> p[PER];
  __device__ __forceinline__ void load(const HeadRows<T, PK>& h, int t0, int ch0, int tid) {
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int x = tid + i * NT;
      if (N % NT == 0 || x < N) p[i] = h.load(t0 + x / PPR, ch0 + (x % PPR) * Lin<T>::EPP);
    }
  }
  __device__ __forceinline__ void store(const HeadRows<T, PK>& h, T* lds, int ld, int tid) const {
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int x = tid + i * NT;
      if (N % NT == 0 || x < N)
        *reinterpret_cast<u32x4_t*>(lds + (x / PPR) * ld + (x % PPR) * Lin<T>::EPP) = p[i].elems(h.packed);
    }
  }
};

// ------------------------------------------------------------------ decay
// a^n for n >= 0 as hi + lo: the chunk factor multiplies the state once per chunk, and a bias of one
// fp32 rounding would add up over the hundreds of chunks of a long sequence.
struct Decay2 {
  float hi, lo;
};
__device__ __forceinline__ Decay2 decay_pow2(float g, int n) {
  const double x = n == 0 ? 1.0 : exp((double)g * n);
  Decay2 d;
  d.hi = (float)x;
  d.lo = (float)(x - (double)d.hi);
  return d;
}
// a^n, g2 = log2(a); n = 0 gives 1 also for a = 0 (g2 = -inf)
__device__ __forceinline__ float decay_pow(float g2, int n) { return n == 0 ? 1.0f : fast_exp2(g2 * (float)n); }

// ------------------------------------------------------------------ state part of a chunk
// The accumulators of one state wave: rows of the channel tiles ct0 .. ct0 + NK - 1, columns of
// the NV value tiles from vt0.
template <typename T, int C, int NK, int NV, bool REV> struct StateTile {
  typedef Lin<T> L;
  floatx4 acc[NK][NV];
  float f[C / L::DG][L::DG / 4];                 // u a^(...) of this lane's tokens
  int n_of_f = -1;

  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < NK; ++i)
#pragma unroll
      for (int j = 0; j < NV; ++j) acc[i][j] = zero4();
  }
  __device__ __forceinline__ void load(const float* S, int sk, int sv, int ct0, int col0, int K, int V, int lane) {
#pragma unroll
    for (int i = 0; i < NK; ++i)
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int row = L::row_of(ct0 + i, 4 * (lane >> 4)), col = col0 + 16 * j + (lane & 15);
#pragma unroll
        for (int r = 0; r < 4; ++r)
          acc[i][j][r] = (row + r < K && col < V) ? S[(size_t)(row + r) * sk + (size_t)col * sv] : 0.0f;
      }
  }
  __device__ __forceinline__ void save(float* S, int sk, int sv, int ct0, int col0, int K, int V, int lane) const {
#pragma unroll
    for (int i = 0; i < NK; ++i)
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int row = L::row_of(ct0 + i, 4 * (lane >> 4)), col = col0 + 16 * j + (lane & 15);
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (row + r < K && col < V) S[(size_t)(row + r) * sk + (size_t)col * sv] = acc[i][j][r];
      }
  }
  // [column][channel] image in LDS
  __device__ __forceinline__ void image(T* dst, int ld, int ct0, int col0, int lane) const {
#pragma unroll
    for (int i = 0; i < NK; ++i)
#pragma unroll
      for (int j = 0; j < NV; ++j)
        L::store4(dst + (col0 + 16 * j + (lane & 15)) * ld + L::row_of(ct0 + i, 4 * (lane >> 4)), acc[i][j]);
  }
  // factors of a chunk of n tokens; tokens behind it get 0
  __device__ __forceinline__ void factors(float g2, float u, int n, int lane) {
    if (n == n_of_f) return;
    n_of_f = n;
#pragma unroll
    for (int d = 0; d < C / L::DG; ++d)
#pragma unroll
      for (int e = 0; e < L::DG / 4; ++e) {
        const int i = d * L::DG + L::tok_of(e, lane >> 4);
        f[d][e] = i < n ? u * decay_pow(g2, REV ? i + 1 : n - 1 - i) : 0.0f;
      }
  }
  __device__ __forceinline__ void update(const T* sK, int ldk, const T* sV, int ldv, int ct0, int vt0, Decay2 an,
                                         int lane) {
#pragma unroll
    for (int i = 0; i < NK; ++i)
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[i][j][r] = fmaf(acc[i][j][r], an.hi, acc[i][j][r] * an.lo);
#pragma unroll
    for (int d = 0; d < C / L::DG; ++d) {
      typename L::frag vf[NV][L::SPLIT];
#pragma unroll
      for (int j = 0; j < NV; ++j)
        L::scaled(L::template tr<false>(sV, ldv, vt0 + j, d * L::DG, lane), f[d], vf[j]);
#pragma unroll
      for (int i = 0; i < NK; ++i) {
        const typename L::frag kf = L::template tr<true>(sK, ldk, ct0 + i, d * L::DG, lane);
#pragma unroll
        for (int s = 0; s < L::SPLIT; ++s)
#pragma unroll
          for (int j = 0; j < NV; ++j) acc[i][j] = L::mma(kf, vf[j][s], acc[i][j]);
      }
    }
  }
};

// ------------------------------------------------------------------ the walk
template <typename T, int KD, int VT, int C> struct WalkShape {
  typedef Lin<T> L;
  static constexpr int LDK = KD + L::PAD, LDV = VT + L::PAD;
  static constexpr int kK = C * LDK, kV = C * LDV, kS = VT * LDK;     // elements
};

// Workgroup -> (head and segment, value tile): the value tiles of one head and segment read the same
// q and k, so they are placed 8 apart, on one XCD (whose L2 then serves the second).
__device__ __forceinline__ void walk_block(int b, int m, int ntile, int* idx, int* tile) {
  const int whole = m / 8 * 8 * ntile;
  if (b < whole) {
    *idx = b / (8 * ntile) * 8 + b % 8;
    *tile = b / 8 % ntile;
  } else {
    *idx = m / 8 * 8 + (b - whole) / ntile;
    *tile = (b - whole) % ntile;
  }
}

template <typename T, int KD, int VT, int C, bool REV, bool PK>
__global__ void __launch_bounds__(512) decay_walk_kernel(WalkArgs a) {
  typedef Lin<T> L;
  typedef WalkShape<T, KD, VT, C> W;
  constexpr int NT = 512;
  constexpr int NTT = C / 16, NVP = 4 / NTT;                 // token tiles; value parts of the output waves
  constexpr int NO = VT / 16 / NVP;                          // value tiles of an output wave
  constexpr int NKS = KD / 32, NVS = VT / 32;                // tiles of a state wave (2 x 2 waves)
  constexpr int NQ = KD / L::DG;
  __shared__ __align__(16) T smem[2 * (W::kK + W::kV + W::kS)];
  static_assert(sizeof(smem) <= 160 * 1024, "LDS of one gfx950 workgroup exceeded");
  T* const sK = smem;
  T* const sV = sK + 2 * W::kK;
  T* const sS = sV + 2 * W::kV;

  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int ntile = (a.V + VT - 1) / VT;
  int idx, tile;
  walk_block(blockIdx.x, a.BH * a.nseg, ntile, &idx, &tile);
  const int bh = idx / a.nseg, seg = idx - bh * a.nseg, v0 = tile * VT;
  const int h = bh % a.H;
  int len = a.T;
  if (a.lengths) len = min(max(a.lengths[bh / a.H], 0), a.T);
  const int t_beg = min(seg * a.seglen, len), t_end = (int)min((long long)seg * a.seglen + a.seglen, (long long)len);
  const int nch = (t_end - t_beg + C - 1) / C;
  const int n_last = t_end - t_beg - (nch - 1) * C;          // tokens of the chunk that may be short
  const float g = a.log_decay[h], g2 = g * kLog2e;

  const HeadRows<T, PK> hq(a.q, a.q_sc, bh, a.T, a.K, t_end), hk(a.k, a.k_sc, bh, a.T, a.K, t_end),
      hv(a.v, a.v_sc, bh, a.T, a.V, t_end);
  const auto chunk_t0 = [&](int ci) { return t_beg + (REV ? nch - 1 - ci : ci) * C; };
  const auto chunk_n = [&](int ci) { return (REV ? ci == 0 : ci == nch - 1) ? n_last : C; };

  const bool is_state = wave >= 4;
  // state waves
  const int sw = wave & 3, ct0 = (sw & 1) * NKS, sv0 = (sw >> 1) * NVS;
  StateTile<T, C, NKS, NVS, REV> st;
  // output waves
  const int ti = wave % NTT, ov0 = (wave & 3) / NTT * NO;
  Piece<T> qn[NQ];
  typename L::frag qf[NQ];
  float pf[NTT][4];
  Decay2 an{0.f, 0.f}, an_short{0.f, 0.f};
  const int tl = 16 * ti + (lane & 15);

  const size_t hs = (size_t)a.K * a.V;
  if (is_state) {
    const float* S0 = a.nseg > 1 ? a.seg_state + ((size_t)bh * a.nseg + seg) * hs
                                 : (a.state_in ? a.state_in + (size_t)bh * hs : nullptr);
    if (S0) st.load(S0, a.si_k, a.si_v, ct0, v0 + 16 * sv0, a.K, a.V, lane);
    else st.zero();
    an = decay_pow2(g, C);
    an_short = decay_pow2(g, nch > 0 ? n_last : 0);
    if (nch > 0) st.image(sS, W::LDK, ct0, 16 * sv0, lane);
  } else {
#pragma unroll
    for (int s = 0; s < NTT; ++s)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int j = 16 * s + 4 * (lane >> 4) + r, d = REV ? j - tl : tl - j;
        pf[s][r] = d < 0 ? 0.0f : a.c * decay_pow(g2, d);
      }
    if (nch > 0) {
#pragma unroll
      for (int x = 0; x < NQ; ++x) qn[x] = hq.load(chunk_t0(0) + tl, x * L::DG + (L::DG / 4) * (lane >> 4));
    }
  }
  Stage<T, PK, C, KD, NT> pk;
  Stage<T, PK, C, VT, NT> pv;
  if (nch > 0) {
    pk.load(hk, chunk_t0(0), 0, tid);
    pv.load(hv, chunk_t0(0), v0, tid);
    pk.store(hk, sK, W::LDK, tid);
    pv.store(hv, sV, W::LDV, tid);
    if (nch > 1) {
      pk.load(hk, chunk_t0(1), 0, tid);
      pv.load(hv, chunk_t0(1), v0, tid);
    }
  }
  lds_barrier();

  T* const oh = reinterpret_cast<T*>(a.o) + (size_t)bh * a.T * a.V;
  const __amdgpu_buffer_rsrc_t ro = make_rsrc(oh, (unsigned)t_end * (unsigned)(a.V * sizeof(T)));

  for (int ci = 0; ci < nch; ++ci) {
    const int cur = ci & 1, n = chunk_n(ci), t0 = chunk_t0(ci);
    const T* cK = sK + cur * W::kK;
    const T* cV = sV + cur * W::kV;
    if (is_state) {
      st.factors(g2, a.u, n, lane);
      st.update(cK, W::LDK, cV, W::LDV, ct0, sv0, n == C ? an : an_short, lane);
      if (ci + 1 < nch) st.image(sS + (cur ^ 1) * W::kS, W::LDK, ct0, 16 * sv0, lane);
    } else {
#pragma unroll
      for (int x = 0; x < NQ; ++x) qf[x] = __builtin_bit_cast(typename L::frag, qn[x].elems(hq.packed));
      if (ci + 1 < nch) {
#pragma unroll
        for (int x = 0; x < NQ; ++x) qn[x] = hq.load(chunk_t0(ci + 1) + tl, x * L::DG + (L::DG / 4) * (lane >> 4));
      }
      const T* cS = sS + cur * W::kS;
      floatx4 acc[NO];
#pragma unroll
      for (int j = 0; j < NO; ++j) acc[j] = zero4();
      // O^T = S^T Q, scaled by the token's read factor (the token is the lane's column)
#pragma unroll
      for (int x = 0; x < NQ; ++x)
#pragma unroll
        for (int j = 0; j < NO; ++j)
          acc[j] = L::mma(L::nat(cS + L::row_of(ov0 + j, lane & 15) * W::LDK, x * L::DG, lane), qf[x], acc[j]);
      const int e = REV ? n - 1 - tl : tl + 1;
      const float rf = a.r * decay_pow(g2, e < 0 ? 0 : e);
#pragma unroll
      for (int j = 0; j < NO; ++j) acc[j] *= rf;
      // scores (keys x tokens) of the tiles the mask reaches, then O^T += V^T scores
#pragma unroll
      for (int d = 0; d < C / L::DG; ++d) {
        const int s0 = d * L::NACC;
        if (REV ? s0 + L::NACC - 1 >= ti : s0 <= ti) {
          floatx4 p[L::NACC];
#pragma unroll
          for (int s = 0; s < L::NACC; ++s) {
            p[s] = zero4();
            if (REV ? s0 + s >= ti : s0 + s <= ti) {
#pragma unroll
              for (int x = 0; x < NQ; ++x)
                p[s] = L::mma(L::nat(cK + (16 * (s0 + s) + (lane & 15)) * W::LDK, x * L::DG, lane), qf[x], p[s]);
#pragma unroll
              for (int r = 0; r < 4; ++r) p[s][r] *= pf[s0 + s][r];
            }
          }
          // scores are rounded to bf16 for the product (fp32 walks keep them): one rounding, 2^-9
          const typename L::frag b = L::from_acc(p);
#pragma unroll
          for (int j = 0; j < NO; ++j)
            acc[j] = L::mma(L::template tr<true>(cV, W::LDV, ov0 + j, d * L::DG, lane), b, acc[j]);
        }
      }
      const unsigned row = (unsigned)(t0 + tl) * (unsigned)(a.V * sizeof(T));
#pragma unroll
      for (int j = 0; j < NO; j += L::NACC) {
        const int col = v0 + L::row_of(ov0 + j, 4 * (lane >> 4));
        const unsigned off = col < a.V ? row + (unsigned)(col * sizeof(T)) : 0xfffffff0u;
        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4_t, L::from_acc(acc + j)), ro, off, 0, 0);
      }
    }
    if (ci + 1 < nch) {
      pk.store(hk, sK + (cur ^ 1) * W::kK, W::LDK, tid);
      pv.store(hv, sV + (cur ^ 1) * W::kV, W::LDV, tid);
      if (ci + 2 < nch) {
        pk.load(hk, chunk_t0(ci + 2), 0, tid);
        pv.load(hv, chunk_t0(ci + 2), v0, tid);
      }
      lds_barrier();
    }
  }
  if (is_state && a.state_out && seg == (REV ? 0 : a.nseg - 1))
    st.save(a.state_out + (size_t)bh * hs, a.si_k, a.si_v, ct0, v0 + 16 * sv0, a.K, a.V, lane);
  if (a.zero_tail) {
    const int e_end = (int)min((long long)seg * a.seglen + a.seglen, (long long)a.T);
    const int e_beg = max(len, seg * a.seglen);
    const int w = min(VT, a.V - v0) / L::EPP;                // 16-byte pieces of a row
    for (long long x = tid; x < (long long)(e_end - e_beg) * w; x += NT)
      *reinterpret_cast<u32x4_t*>(oh + (size_t)(e_beg + x / w) * a.V + v0 + (x % w) * L::EPP) = u32x4_t{0, 0, 0, 0};
  }
}

// Local end state of every segment but the last in walking order.
template <typename T, int KD, int VT, int C, bool REV, bool PK>
__global__ void __launch_bounds__(256) decay_segment_kernel(SegArgs a) {
  typedef WalkShape<T, KD, VT, C> W;
  constexpr int NT = 256, NKS = KD / 32, NVS = VT / 32;
  __shared__ __align__(16) T smem[2 * (W::kK + W::kV)];
  T* const sK = smem;
  T* const sV = sK + 2 * W::kK;
  const int tid = threadIdx.x, lane = tid & 63, sw = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int ntile = (a.V + VT - 1) / VT;
  int idx, tile;
  walk_block(blockIdx.x, a.BH * (a.nseg - 1), ntile, &idx, &tile);
  const int bh = idx / (a.nseg - 1), seg = idx - bh * (a.nseg - 1) + (REV ? 1 : 0), v0 = tile * VT;
  int len = a.T;
  if (a.lengths) len = min(max(a.lengths[bh / a.H], 0), a.T);
  const int t_beg = min(seg * a.seglen, len), t_end = (int)min((long long)seg * a.seglen + a.seglen, (long long)len);
  const int nch = (t_end - t_beg + C - 1) / C;
  const int n_last = t_end - t_beg - (nch - 1) * C;
  const float g = a.log_decay[bh % a.H], g2 = g * kLog2e;
  const HeadRows<T, PK> hk(a.k, a.k_sc, bh, a.T, a.K, t_end), hv(a.v, a.v_sc, bh, a.T, a.V, t_end);
  const auto chunk_t0 = [&](int ci) { return t_beg + (REV ? nch - 1 - ci : ci) * C; };
  const auto chunk_n = [&](int ci) { return (REV ? ci == 0 : ci == nch - 1) ? n_last : C; };
  const int ct0 = (sw & 1) * NKS, sv0 = (sw >> 1) * NVS;
  StateTile<T, C, NKS, NVS, REV> st;
  st.zero();
  const Decay2 an = decay_pow2(g, C), an_short = decay_pow2(g, nch > 0 ? n_last : 0);
  Stage<T, PK, C, KD, NT> pk;
  Stage<T, PK, C, VT, NT> pv;
  if (nch > 0) {
    pk.load(hk, chunk_t0(0), 0, tid);
    pv.load(hv, chunk_t0(0), v0, tid);
  }
  for (int ci = 0; ci < nch; ++ci) {
    const int cur = ci & 1, n = chunk_n(ci);
    // the buffer written here was last read two chunks ago, before the previous barrier
    pk.store(hk, sK + cur * W::kK, W::LDK, tid);
    pv.store(hv, sV + cur * W::kV, W::LDV, tid);
    if (ci + 1 < nch) {
      pk.load(hk, chunk_t0(ci + 1), 0, tid);
      pv.load(hv, chunk_t0(ci + 1), v0, tid);
    }
    lds_barrier();
    st.factors(g2, a.u, n, lane);
    st.update(sK + cur * W::kK, W::LDK, sV + cur * W::kV, W::LDV, ct0, sv0, n == C ? an : an_short, lane);
  }
  st.save(a.seg_state + ((size_t)bh * a.nseg + seg) * a.K * a.V, a.V, 1, ct0, v0 + 16 * sv0, a.K, a.V, lane);
}

// ------------------------------------------------------------------ launchers
template <typename T> constexpr int walk_chunk() { return std::is_same<T, float>::value ? 32 : 64; }

template <typename T, int KD, int VT, bool REV, bool PK>
hipError_t launch_walk_inst(const WalkArgs& a, hipStream_t s) {
  constexpr int C = walk_chunk<T>();
  const auto kern = decay_walk_kernel<T, KD, VT, C, REV, PK>;
  const int blocks = a.BH * a.nseg * ((a.V + VT - 1) / VT);
  hipLaunchKernelGGL(kern, dim3(blocks), dim3(512), 0, s, a);
  return hipGetLastError();
}

template <typename T, int KD, int VT, bool REV, bool PK>
hipError_t launch_segments_inst(const SegArgs& a, hipStream_t s) {
  constexpr int C = walk_chunk<T>();
  const auto kern = decay_segment_kernel<T, KD, VT, C, REV, PK>;
  const int blocks = a.BH * (a.nseg - 1) * ((a.V + VT - 1) / VT);
  hipLaunchKernelGGL(kern, dim3(blocks), dim3(256), 0, s, a);
  return hipGetLastError();
}

// Instances by padded key width KD; the value tile is 64 columns, or 32 where V <= 32.
template <typename T, int KD, bool PK>
hipError_t launch_walk_kd(const WalkArgs& a, bool rev, hipStream_t s) {
  if (a.V <= 32) return rev ? launch_walk_inst<T, KD, 32, true, PK>(a, s) : launch_walk_inst<T, KD, 32, false, PK>(a, s);
  return rev ? launch_walk_inst<T, KD, 64, true, PK>(a, s) : launch_walk_inst<T, KD, 64, false, PK>(a, s);
}
template <typename T, int KD, bool PK>
hipError_t launch_segments_kd(const SegArgs& a, bool rev, hipStream_t s) {
  if (a.V <= 32)
    return rev ? launch_segments_inst<T, KD, 32, true, PK>(a, s) : launch_segments_inst<T, KD, 32, false, PK>(a, s);
  return rev ? launch_segments_inst<T, KD, 64, true, PK>(a, s) : launch_segments_inst<T, KD, 64, false, PK>(a, s);
}

}  // namespace kda
