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
// eight waves in two roles.  State waves hold S (KD x VT, fp32) in accumulators, 16 value columns each, and
// leave its bf16 (or fp32) image in LDS for the next chunk; output waves each own 16 tokens: their
// scores K Q^T come out of the matrix unit in the layout in which the product with V takes them, so
// the scores never touch LDS.  The roles overlap on every SIMD and meet at one barrier per chunk.
//
// What bounds it: 4 x 32 heads of 16384 tokens, K = V = 128, bf16: 446 to 458 us for 2.16 GB, 4.7 to 4.85 TB/s, the rate
// of a large copy, at a socket power of 1395 W and clocks held at 1.65 GHz.  Shorter ones: the chain of a chunk in two in-order waves per SIMD, 1.05 us per 64 tokens at K = V = 64 (with
// only the output or only the state waves at work 0.87 and 0.84) and 1.4 us at 128, where the matrix unit's share is
// 0.45 and the LDS is busy for a third.  fp32 (1 x 16 heads of 8191, K = V = 128, backward, 425 us) has the matrix unit
// busy for 71 % of the walk's cycles.
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
  float* mid;                // null, or takes the states at the starts of nmid segments of midlen tokens that
  int nmid, midlen;          // another walk is cut into (reverse walks of one segment; same strides)
  void* o;
  float c, r, u;             // scales of the intra-chunk term, the read and the update
  int si_k, si_v;
  int BH, H, T, K, V;        // K, V: the walk's key and value widths
  int nseg, seglen;          // seglen: a multiple of the chunk
  int returned;              // the state, or one that follows from it, is returned (see fine_state)
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
  bool returned;             // the end state that these lead to is returned
};

typedef unsigned int u32x4_t __attribute__((ext_vector_type(4)));
typedef unsigned int u32x2_t __attribute__((ext_vector_type(2)));
typedef short short4v_t __attribute__((ext_vector_type(4)));

// Pointers into LDS keep their address space (a generic one would be tested for null at every cast).
template <typename U> using Lds = __attribute__((address_space(3))) U;

// ------------------------------------------------------------------ operand layouts
// A product's contraction runs in groups of DG indices.  A fragment holds, for row (or column)
// lane % 16 and lane group g = lane / 16, DG / 4 of the group's indices: DG / 4 consecutive ones
// when read along memory (`nat`), or those in which NACC accumulator tiles hold them (`from_acc`:
// index 16 n + 4 g + r of tile n).  `tr` reads the transpose of a [index][column] tile in the
// accumulator order.  Tile `ct` of 16 rows covers the rows row_of(ct, m), m = 0..15: a lane's accumulator
// registers hold four consecutive rows of each, and of NACC adjacent tiles DG / 4 consecutive rows.
//
// LDS has 64 banks of 4 bytes.  One cycle serves 16 lanes of a 16-byte read, and these are not consecutive:
// lanes 0-3, 12-15 and 20-27 of each 32, then the others (of a natural read, rows 0-3 and 12-15 at one piece
// and rows 4-11 at the next); 32 consecutive lanes of an 8-byte read, 16 of an 8-byte write (measured, two
// lanes at a time).  bf16 tiles are [row][W elements] without padding; the 16-byte pieces of row t are stored
// in the order piece ^ swz(t).  64 banks hold 16 pieces, so W's pieces per row leave some low bits of t to
// the address and the rest to swz, whose lowest bit differs between two rows of 4-11 (and of the others).
// With row_of()'s halves, which alternate from one lane group to the next, every read above and the image's
// writes then fall on different banks.  (Rows padded by 16 bytes, and rows in the order piece ^ t, took
// twice the cycles for every one of these reads.)  fp32 rows are padded by 16 bytes: their transposed
// reads are single words, free of conflicts; natural reads take two cycles for one.
template <typename T> struct Lin;

template <> struct Lin<bf16_t> {                 // v_mfma_f32_16x16x32_bf16
  static constexpr int DG = 32, NACC = 2, EPP = 8, PAD = 0, PARTS = 2;
  typedef short8 frag;
  static __device__ __forceinline__ int row_of(int ct, int m) {
    return 32 * (ct >> 1) + 8 * (m >> 2) + 4 * ((ct ^ m >> 2) & 1) + (m & 3);
  }
  // IMG: the state image, whose natural reads take the rows row_of() of a tile
  template <int W, bool IMG> static __device__ __forceinline__ int swz(int t) {
    const int lo = IMG ? ((t >> 4 ^ t >> 2) & 1) << 1 | (t >> 3 & 1) : ((t >> 3 ^ t >> 2) & 1) << 1 | (t >> 2 & 1);
    if constexpr (W == 128) return (t & 3) << 2 | lo;
    else if constexpr (W == 64) return (t & 2) << 1 | lo;
    else return lo;
  }
  template <int W, bool IMG> static __device__ __forceinline__ int at(int t, int e) {
    return t * W + ((e >> 3) ^ swz<W, IMG>(t)) * 8 + (e & 7);
  }
  template <int W, bool IMG>
  static __device__ __forceinline__ frag nat(const Lds<bf16_t>* base, int t, int d0, int lane) {
    return *(const Lds<short8>*)(base + at<W, IMG>(t, d0 + 8 * (lane >> 4)));
  }
  // two transposing reads: lane 4r + m of a group of 16 addresses row 4g + r (then 16 + 4g + r) at
  // four columns and lane j receives column j of the group's 16
  template <int W, bool PERM> static __device__ __forceinline__ frag tr(const Lds<bf16_t>* base, int ct, int d0, int lane) {
    const int g = lane >> 4, r = (lane >> 2) & 3, m = lane & 3;
    const int col = PERM ? row_of(ct, 4 * m) : 16 * ct + 4 * m;
    const Lds<bf16_t>* p = base + at<W, false>(d0 + 4 * g + r, col);     // (swz is the same 16 rows on)
    const short4v_t a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((Lds<short4v_t>*)p);
    const short4v_t b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((Lds<short4v_t>*)(p + 16 * W));
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
  // the 8 consecutive rows that a lane holds of tiles ct, ct + 1 (ct even): in odd lane groups the second
  // tile has the first four
  static __device__ __forceinline__ u32x4_t row16(const floatx4* x, int lane) {
    const u32x2_t a = {pack_bf16x2(x[0][0], x[0][1]), pack_bf16x2(x[0][2], x[0][3])};
    const u32x2_t b = {pack_bf16x2(x[1][0], x[1][1]), pack_bf16x2(x[1][2], x[1][3])};
    const bool odd = lane >> 4 & 1;
    return u32x4_t{odd ? b[0] : a[0], odd ? b[1] : a[1], odd ? a[0] : b[0], odd ? a[1] : b[1]};
  }
  // x f as bf16 parts: the sum of the first two is off by at most 2^-17 of it, with the third 2^-26
  static __device__ __forceinline__ void scaled(frag x, const float* f, frag* out) {
    u32x4_t part[2];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float a = bf2f((bf16_t)x[2 * e]) * f[2 * e], b = bf2f((bf16_t)x[2 * e + 1]) * f[2 * e + 1];
      const uint32_t w = pack_bf16x2(a, b);
      part[0][e] = w;
      part[1][e] = pack_bf16x2(a - __uint_as_float(w << 16), b - __uint_as_float(w & 0xffff0000u));
    }
    out[0] = __builtin_bit_cast(short8, part[0]);
    out[1] = __builtin_bit_cast(short8, part[1]);
  }
  static __device__ __forceinline__ frag third(frag x, const float* f) {
    u32x4_t part;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float a = bf2f((bf16_t)x[2 * e]) * f[2 * e], b = bf2f((bf16_t)x[2 * e + 1]) * f[2 * e + 1];
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const uint32_t w = pack_bf16x2(a, b);
        a -= __uint_as_float(w << 16);
        b -= __uint_as_float(w & 0xffff0000u);
      }
      part[e] = pack_bf16x2(a, b);
    }
    return __builtin_bit_cast(short8, part);
  }
  // token (within a group of DG) of fragment element e in the accumulator order
  static __device__ __forceinline__ int tok_of(int e, int g) { return 16 * (e >> 2) + 4 * g + (e & 3); }
  static __device__ __forceinline__ void store4(Lds<bf16_t>* p, floatx4 x) {
    *(Lds<u32x2_t>*)p = u32x2_t{pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3])};
  }
};

template <> struct Lin<float> {                  // four v_mfma_f32_16x16x4_f32
  static constexpr int DG = 16, NACC = 1, EPP = 4, PAD = 4, PARTS = 1;
  typedef floatx4 frag;
  static __device__ __forceinline__ int row_of(int ct, int m) { return 16 * ct + m; }
  template <int W, bool IMG> static __device__ __forceinline__ int at(int t, int e) { return t * (W + PAD) + e; }
  template <int W, bool IMG>
  static __device__ __forceinline__ frag nat(const Lds<float>* base, int t, int d0, int lane) {
    return *(const Lds<floatx4>*)(base + at<W, IMG>(t, d0 + 4 * (lane >> 4)));
  }
  template <int W, bool PERM> static __device__ __forceinline__ frag tr(const Lds<float>* base, int ct, int d0, int lane) {
    const int t = d0 + 4 * (lane >> 4), e = 16 * ct + (lane & 15);
    return floatx4{base[at<W, false>(t, e)], base[at<W, false>(t + 1, e)], base[at<W, false>(t + 2, e)],
                   base[at<W, false>(t + 3, e)]};
  }
  static __device__ __forceinline__ floatx4 mma(frag a, frag b, floatx4 c) {
#pragma unroll
    for (int r = 0; r < 4; ++r) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[r], b[r], c, 0, 0, 0);
    return c;
  }
  static __device__ __forceinline__ frag from_acc(const floatx4* x) { return x[0]; }
  static __device__ __forceinline__ u32x4_t row16(const floatx4* x, int) { return __builtin_bit_cast(u32x4_t, x[0]); }
  static __device__ __forceinline__ void scaled(frag x, const float* f, frag* out) {
    out[0] = floatx4{x[0] * f[0], x[1] * f[1], x[2] * f[2], x[3] * f[3]};
  }
  static __device__ __forceinline__ int tok_of(int e, int g) { return 4 * g + e; }
  static __device__ __forceinline__ void store4(Lds<float>* p, floatx4 x) { *(Lds<floatx4>*)p = x; }
};

// ------------------------------------------------------------------ loads
// 2^(b - 127) for a scale byte b (b = 0: 2^-127, a subnormal).
__device__ __forceinline__ float ckpt_scale(uint32_t b) { return __uint_as_float(b ? b << 23 : 0x00400000u); }

// One piece of EPP consecutive channels of a row on its way from memory: 16 bytes of elements, or (PK)
// EPP codes and their group's scale byte.
template <typename T, bool PK> struct Piece {
  static constexpr int W = PK ? Lin<T>::EPP / 4 : 4;
  uint32_t raw[W];
  uint32_t sc;
  __device__ __forceinline__ u32x4_t elems() const {
    if constexpr (!PK) {
      return u32x4_t{raw[0], raw[1], raw[2], raw[3]};
    } else {
      const float s = ckpt_scale(sc);
      float f[4 * W];
#pragma unroll
      for (int i = 0; i < W; ++i) {
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
  }
};

// Words of a raw buffer resource, for the copies below.
__device__ __forceinline__ u32x4_t buffer_words(const void* base, unsigned bytes) {
  const uintptr_t p = (uintptr_t)base;
  return u32x4_t{(uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)p),
                 (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(p >> 32)) & 0xffffu,
                 (uint32_t)__builtin_amdgcn_readfirstlane((int)bytes), 0x00020000u};
}
// One head of a tensor (rows tokens x D channels) behind a range-checked buffer: rows from `len` on
// and channels from D on read as zero.
template <typename T, bool PK> struct HeadRows {
  __amdgpu_buffer_rsrc_t r, rs;
  u32x4_t words;                                 // of r, for the copies
  int D, nsc;
  __device__ __forceinline__ HeadRows(const void* base, const uint8_t* sc, int bh, int T_, int D_, int len) {
    D = D_;
    constexpr int es = PK ? 1 : (int)sizeof(T);
    const char* head = (const char*)base + (size_t)bh * T_ * D * es;
    r = make_rsrc(head, (unsigned)len * (unsigned)(D * es));
    words = buffer_words(head, (unsigned)len * (unsigned)(D * es));
    nsc = D < 32 ? 1 : D / 32;
    if constexpr (PK) rs = make_rsrc(sc + (size_t)bh * T_ * nsc, (unsigned)len * (unsigned)nsc);
  }
  __device__ __forceinline__ Piece<T, PK> load(int t, int ch) const {
    Piece<T, PK> p;
    constexpr unsigned kOut = 0xfffffff0u;                     // past any buffer's range
    const unsigned at = (unsigned)t * (unsigned)D + (unsigned)ch;
    const bool in = ch < D;
    if constexpr (!PK) {
      const u32x4_t x = __builtin_bit_cast(
          u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(r, in ? at * (unsigned)sizeof(T) : kOut, 0, 0));
#pragma unroll
      for (int i = 0; i < 4; ++i) p.raw[i] = x[i];
    } else {
      if constexpr (Piece<T, PK>::W == 1) {
        p.raw[0] = __builtin_amdgcn_raw_buffer_load_b32(r, in ? at : kOut, 0, 0);
      } else {
        const u32x2_t x =
            __builtin_bit_cast(u32x2_t, __builtin_amdgcn_raw_buffer_load_b64(r, in ? at : kOut, 0, 0));
        p.raw[0] = x[0];
        p.raw[1] = x[1];
      }
      p.sc = __builtin_amdgcn_raw_buffer_load_b8(
          rs, in ? (unsigned)t * (unsigned)nsc + (unsigned)(ch >> 5) : kOut, 0, 0);
    }
    return p;
  }
};

// LDS image of C rows x DP channels: row pitch and size in 16-byte pieces (a size that whole waves fill).
template <typename T, int C, int DP> struct Tile {
  static constexpr int PPR = (DP + Lin<T>::PAD) / Lin<T>::EPP, NP = round_up(C * PPR, 64), ELEMS = NP * Lin<T>::EPP;
};

// A chunk of C rows x DP channels (from ch0) held by the NT threads between memory and LDS (8-bit
// operands, whose codes become elements on the way).
template <typename T, bool PK, int C, int DP, int NT> struct Stage {
  static constexpr int PPR = DP / Lin<T>::EPP, N = C * PPR, PER = (N + NT - 1) / NT;
  Piece<T, PK> p[PER];
  __device__ __forceinline__ void load(const HeadRows<T, PK>& h, int t0, int ch0, int tid) {
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int x = tid + i * NT;
      if (N % NT == 0 || x < N) p[i] = h.load(t0 + x / PPR, ch0 + (x % PPR) * Lin<T>::EPP);
    }
  }
  __device__ __forceinline__ void store(Lds<T>* lds, int tid) const {
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int x = tid + i * NT;
      if (N % NT == 0 || x < N)
        *(Lds<u32x4_t>*)(lds + Lin<T>::template at<DP, false>(x / PPR, (x % PPR) * Lin<T>::EPP)) =
            p[i].elems();
    }
  }
};

// 16 bytes per lane from byte `lane_off` + `off` of the buffer into LDS at lds + 16 * lane (lds and off are
// the wave's).  Past the buffer's range: zeros.  Written in asm, with no register as its output, because
// the compiler would wait for every copy in flight before each transposing LDS read; the waits are
// wait_vm_but()'s (the compiler's own waits for its loads and stores only grow stricter by operations that
// it does not count).  Nor does the compiler look into the block for hazards, so the block holds the wait states
// itself, whatever stands in front of it: one between m0's write and its use, and five between a vector instruction
// that writes a scalar register (a readlane of a spilled one, a readfirstlane) and a copy that reads it: the move
// to m0 and the four of s_nop 3.
__device__ __forceinline__ void copy_to_lds(u32x4_t r, const Lds<void>* lds, unsigned lane_off, unsigned off) {
  const uint32_t at = (uint32_t)(uintptr_t)lds;
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 3\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds" ::"s"(
                   __builtin_amdgcn_readfirstlane((int)at)),
               "v"(lane_off), "s"(r), "s"(off)
               : "memory", "m0");
}

// Byte offset, from a tile's first row (channels from ch0, D in a row), of the 16-byte piece that belongs into
// place `slot` of the tile's LDS image of C rows x DP channels; past any range for the places of its padding.
template <typename T, int C, int DP> __device__ __forceinline__ unsigned copy_offset(int slot, int D, int ch0) {
  typedef Tile<T, C, DP> TL;
  constexpr int E = Lin<T>::EPP;
  const int row = slot / TL::PPR, pos = slot % TL::PPR;
  int pc = pos;
  if constexpr (Lin<T>::PAD == 0) pc = pos ^ (Lin<T>::template at<DP, false>(row, 0) - row * DP) / E;
  const int ch = ch0 + pc * E;
  return row < C && pc < DP / E && ch < D ? (unsigned)(row * D + ch) * (unsigned)sizeof(T) : 0xfffffff0u;
}

// A tile copied from memory straight into LDS: each wave instruction fills 64 consecutive pieces, so the
// order of the pieces within a row is made by the address each lane reads.  Rows behind the range read as
// zeros.  bf16 rows repeat their order every 16, so a tile's instructions share PERIOD lane offsets and
// differ by a scalar one.
template <typename T, int C, int DP> struct CopyTile {
  typedef Tile<T, C, DP> TL;
  static constexpr int E = Lin<T>::EPP, N = TL::NP / 64;       // N instructions
  static constexpr int PERIOD = Lin<T>::PAD == 0 ? cmax(1, 16 * TL::PPR / 64) : N;
  unsigned off[PERIOD], row_bytes;
  __device__ __forceinline__ CopyTile(int lane, int D, int ch0) {
    row_bytes = (unsigned)(D * (int)sizeof(T));
#pragma unroll
    for (int i = 0; i < PERIOD; ++i) off[i] = copy_offset<T, C, DP>(64 * i + lane, D, ch0);
  }
  // instruction I of the tile whose first row is token t0
  template <int I> __device__ __forceinline__ void issue(u32x4_t r, int t0, const Lds<T>* lds) const {
    constexpr unsigned rows = I / PERIOD * (PERIOD * 64 / TL::PPR);
    copy_to_lds(r, lds + I * 64 * E, off[I % PERIOD], ((unsigned)t0 + rows) * row_bytes);
  }
  template <int I0, int I1> __device__ __forceinline__ void issue_range(u32x4_t r, int t0, const Lds<T>* lds) const {
    if constexpr (I0 < I1) {
      issue<I0>(r, t0, lds);
      issue_range<I0 + 1, I1>(r, t0, lds);
    }
  }
};
// The k and v tiles of one chunk by all NW waves of a workgroup, MIN or MIN + 1 instructions each.
template <typename T, int C, int DK, int DV, int NW> struct Copy {
  static constexpr int IK = Tile<T, C, DK>::NP / 64, IV = Tile<T, C, DV>::NP / 64, NI = IK + IV;
  static constexpr int PER = (NI + NW - 1) / NW, MIN = NI / NW;
  unsigned off[PER];                             // byte offset of this lane's piece from the chunk's first row

  __device__ __forceinline__ Copy(int wave, int lane, int K, int V, int v0) {
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int x = wave + i * NW;
      off[i] = x < IK ? copy_offset<T, C, DK>(64 * x + lane, K, 0) : copy_offset<T, C, DV>(64 * (x - IK) + lane, V, v0);
    }
  }
  // tokens from t0 into the tiles at lds (v behind k)
  __device__ __forceinline__ void issue(u32x4_t rk, u32x4_t rv, int t0, int K, int V, const Lds<T>* lds,
                                        int wave) const {
    const unsigned sk = (unsigned)t0 * (unsigned)(K * sizeof(T)), sv = (unsigned)t0 * (unsigned)(V * sizeof(T));
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int x = wave + i * NW;
      if (NI % NW == 0 || x < NI) copy_to_lds(x < IK ? rk : rv, lds + x * 64 * Lin<T>::EPP, off[i], x < IK ? sk : sv);
    }
  }
};
// Until at most N of this wave's latest vector-memory operations are outstanding.
template <int N> __device__ __forceinline__ void wait_vm_but() { asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory"); }
// Until none is, known to the compiler too: before a loop with copies in flight, so that it does not wait in
// the loop for loads from before it.
__device__ __forceinline__ void wait_vm_all() { __builtin_amdgcn_s_waitcnt(0x0F70); }
// Barrier for LDS that leaves copies into LDS in flight: each wave waits for its own reads and writes, and
// before it for the copies that the next chunk needs.
__device__ __forceinline__ void chunk_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// ------------------------------------------------------------------ decay
// A value that is the same in all lanes, kept in a scalar register.
__device__ __forceinline__ float uniform(float x) {
  return __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(x)));
}

// a^n for n >= 0, once per walk.
__device__ __forceinline__ double decay_pow64(float g, int n) { return n == 0 ? 1.0 : exp((double)g * n); }
__device__ __forceinline__ float decay_pow32(float g, int n) { return uniform((float)decay_pow64(g, n)); }
// The factors a^n of equal steps of n tokens, by which a state goes from one chunk (or segment) to the next.  a^n
// rounded to fp32 is off by up to half a place, and to the same side in each of the thousands of chunks of a long
// sequence (6e-5 after 2048 of them).  So what one factor is off by is owed to the next, and the product of any run
// of them is off by one place.  (Adding lo x to the rounded product hi x does nothing, as it is below half of x's
// last place.  Both in one rounding, fma(x, hi, x lo), is as exact; fp32 walks took 3.5 % longer with it.)
struct DecaySteps {
  float hi, lo, owed;
  __device__ __forceinline__ DecaySteps(float g, int n) {
    const double x = decay_pow64(g, n);
    const float h = (float)x;
    hi = uniform(h), lo = uniform((float)(x - (double)h)), owed = 0.0f;
  }
  __device__ __forceinline__ float next() {
    owed += lo;
    const float m = hi + owed;
    owed = uniform(owed - (m - hi));
    return m;
  }
};
// a^n, g2 = log2(a); n = 0 gives 1 also for a = 0 (g2 = -inf)
__device__ __forceinline__ float decay_pow(float g2, int n) { return n == 0 ? 1.0f : fast_exp2(g2 * (float)n); }


// ------------------------------------------------------------------ state part of a chunk
// The accumulators of one state wave: rows of the channel tiles ct0 .. ct0 + NK - 1, columns of
// the NV value tiles from vt0.
template <typename T, int KD, int VT, int C, int NK, int NV, bool REV> struct StateTile {
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
        // (rows and columns of the padding: some element of the state, then zero)
        const int row = L::row_of(ct0 + i, 4 * (lane >> 4)), col = col0 + 16 * j + (lane & 15);
        const bool in = row < K && col < V;                  // K is a multiple of 4
        const float* p = S + (in ? row * sk + col * sv : 0);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float x = p[r * sk];
          acc[i][j][r] = in ? x : 0.0f;
        }
      }
  }
  __device__ __forceinline__ void save(float* S, int sk, int sv, int ct0, int col0, int K, int V, int lane) const {
#pragma unroll
    for (int i = 0; i < NK; ++i)
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int row = L::row_of(ct0 + i, 4 * (lane >> 4)), col = col0 + 16 * j + (lane & 15);
        if (row < K && col < V) {
          float* p = S + row * sk + col * sv;
#pragma unroll
          for (int r = 0; r < 4; ++r) p[r * sk] = acc[i][j][r];
        }
      }
  }
  // [column][channel] image in LDS
  __device__ __forceinline__ void image(Lds<T>* dst, int ct0, int col0, int lane) const {
#pragma unroll
    for (int i = 0; i < NK; ++i)
#pragma unroll
      for (int j = 0; j < NV; ++j)
        L::store4(dst + L::template at<KD, true>(col0 + 16 * j + (lane & 15), L::row_of(ct0 + i, 4 * (lane >> 4))),
                  acc[i][j]);
  }
  // factors of a chunk of n tokens; tokens behind it get 0
  __device__ __forceinline__ void factors(float g2, float u, int n, int lane) {
    if (n == n_of_f) return;
    n_of_f = n;
    asm volatile("" : "+v"(lane));                 // computed here, not kept from before the loop
#pragma unroll
    for (int d = 0; d < C / L::DG; ++d)
#pragma unroll
      for (int e = 0; e < L::DG / 4; ++e) {
        const int i = d * L::DG + L::tok_of(e, lane >> 4);
        f[d][e] = i < n ? u * decay_pow(g2, REV ? i + 1 : n - 1 - i) : 0.0f;
      }
  }
  // a: the chunk's decay; `fine`: the products as exactly as fp32 holds them (see fine_state)
  __device__ __forceinline__ void update(const Lds<T>* sK, const Lds<T>* sV, int ct0, int vt0, float a, bool fine,
                                         int lane) {
    // bf16: every operand requested at once, the decay behind the requests (8 x 8 heads of 4096 tokens, K = V = 64: 3 %
    // faster); fp32, which has four times the products to hide a request behind, as it is used (2 % faster)
    constexpr int ND = C / L::DG;
    constexpr bool EARLY = L::PARTS > 1;
    typename L::frag v[ND][NV], kf[ND][NK];
    const auto read = [&](int d) {
#pragma unroll
      for (int j = 0; j < NV; ++j) v[d][j] = L::template tr<VT, false>(sV, vt0 + j, d * L::DG, lane);
#pragma unroll
      for (int i = 0; i < NK; ++i) kf[d][i] = L::template tr<KD, true>(sK, ct0 + i, d * L::DG, lane);
    };
    if constexpr (EARLY) {
#pragma unroll
      for (int d = 0; d < ND; ++d) read(d);
    }
#pragma unroll
    for (int i = 0; i < NK; ++i)
#pragma unroll
      for (int j = 0; j < NV; ++j) acc[i][j] *= a;
#pragma unroll
    for (int d = 0; d < ND; ++d) {
      if constexpr (!EARLY) read(d);
      typename L::frag vf[NV][L::PARTS];
#pragma unroll
      for (int j = 0; j < NV; ++j) L::scaled(v[d][j], f[d], vf[j]);
#pragma unroll
      for (int s = 0; s < L::PARTS; ++s)
#pragma unroll
        for (int i = 0; i < NK; ++i)
#pragma unroll
          for (int j = 0; j < NV; ++j) acc[i][j] = L::mma(kf[d][i], vf[j][s], acc[i][j]);
    }
    if constexpr (L::PARTS > 1) {
      if (fine) {
#pragma unroll
        for (int d = 0; d < ND; ++d)
#pragma unroll
          for (int j = 0; j < NV; ++j) {
            const typename L::frag t = L::third(v[d][j], f[d]);
#pragma unroll
            for (int i = 0; i < NK; ++i) acc[i][j] = L::mma(kf[d][i], t, acc[i][j]);
          }
      }
    }
  }
};

// How exactly a bf16 chunk's part of the state is computed (fp32 products need no parts).  The state serves two
// ends.  The outputs read its bf16 image: two bf16 parts of the decayed operand (2^-17) are far below that
// rounding.  The end state is returned in fp32, where they would show (2.8e-6 of the state), but only from chunks
// that the decay to the end leaves something of: a chunk counts as fine, three parts (2^-26), while
// a^{tokens behind it} is over 2^-10, and none does where no end state is returned.  At 4 x 32 heads of 16384
// tokens, K = V = 128, log decays of -0.8 to -0.002, all chunks fine take 500 us, by this rule 459 (the GPU runs this
// walk at its power limit, see above, so time follows the matrix work).
__device__ __forceinline__ bool fine_state(bool returned, float g2, int behind) {
  return returned && !(g2 * (float)behind <= -10.0f);                  // (also for -inf times 0)
}

// ------------------------------------------------------------------ the walk
// How NW state waves share the KD x VT state: one 16-column value tile and a part of the channels each.
template <int KD, int VT, int NW> struct StateShape {
  static constexpr int WV = cmin(VT / 16, NW), WK = NW / WV;
  static constexpr int NK = KD / 16 / WK, NV = VT / 16 / WV;          // tiles of a wave
  static_assert(NK >= 1 && NV >= 1, "tile too small for the waves");
};

constexpr int kWalkThreads = 512;
// Four output waves: one per 16 tokens (and, in fp32's shorter chunks, per half of the value tile).  Four
// state waves of about the same length.
template <typename T, int KD, int VT> struct WalkShape {
  typedef Lin<T> L;
  static constexpr int C = sizeof(T) == 4 ? 32 : 64;
  static constexpr int NTT = C / 16, NVP = 4 / NTT;                   // output waves: token tiles x value parts
  static constexpr int NO = VT / 16 / NVP;                            // value tiles of an output wave
  typedef StateShape<KD, VT, 4> S;
  static_assert(NO >= L::NACC, "tile too small for the waves");
  // waves per SIMD that the registers are cut to, none of which may spill to memory (a spilled operand would be
  // waited for in every chunk): one workgroup of 8 waves per CU for the widest keys, two for narrower ones (of
  // fp32 tiles of 64 x 64, 90 KB, the LDS holds one).
  static constexpr int EU = KD == 128 ? 2 : 4;
  static constexpr int kK = Tile<T, C, KD>::ELEMS, kV = Tile<T, C, VT>::ELEMS, kS = VT * (KD + L::PAD);
  static constexpr int kC = 2 * kK + kV;                              // a chunk's k, v and q
  // chunks in LDS: three (a copy has two chunks' time to arrive) where one workgroup has the CU for
  // itself anyway and they fit
  static constexpr int NS = sizeof(T) * (3 * kC + 2 * kS) <= 160 * 1024 && EU == 2 ? 3 : 2;
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

// LDS elements of a walk; 8-bit operands go through registers and need two chunks only.
template <typename T, int KD, int VT, bool PACK> constexpr int walk_lds() {
  typedef WalkShape<T, KD, VT> W;
  return (PACK ? 2 : W::NS) * W::kC + 2 * W::kS;
}

// PQ, PK, PV: the operand is kept in 8 bits.
template <typename T, int KD, int VT, bool REV, bool PQ, bool PK, bool PV>
__device__ __forceinline__ void walk(const WalkArgs& a, int block, Lds<T>* smem) {
  typedef Lin<T> L;
  typedef typename L::frag frag;
  typedef WalkShape<T, KD, VT> W;
  constexpr int C = W::C, NT = kWalkThreads, NTT = W::NTT, NO = W::NO, NKS = W::S::NK, NVS = W::S::NV;
  constexpr int NQ = KD / L::DG, ND = C / L::DG;
  static_assert(ND == 2, "two groups of tokens per chunk");
  constexpr bool DMA = !(PQ || PK || PV);
  constexpr int NS = DMA ? W::NS : 2;
  Lds<T>* const sS = smem + NS * W::kC;
  // the chunk's place in LDS, kept as an offset in a scalar register (a remainder by NS would be carried
  // through every lane's addresses)
  const auto next_slot = [](unsigned s) {
    s = s == (NS - 1) * W::kC ? 0u : s + (unsigned)W::kC;
    asm volatile("" : "+s"(s));
    return s;
  };
  const auto tile_k = [&](unsigned at) { return smem + at; };
  const auto tile_v = [&](unsigned at) { return smem + at + W::kK; };
  const auto tile_q = [&](unsigned at) { return smem + at + W::kK + W::kV; };

  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int ntile = (a.V + VT - 1) / VT;
  int idx, tile;
  walk_block(block, a.BH * a.nseg, ntile, &idx, &tile);
  const int bh = idx / a.nseg, seg = idx - bh * a.nseg, v0 = tile * VT;
  const int h = bh % a.H;
  int len = a.T;
  if (a.lengths) len = min(max(a.lengths[bh / a.H], 0), a.T);
  const int t_beg = min(seg * a.seglen, len), t_end = (int)min((long long)seg * a.seglen + a.seglen, (long long)len);
  const int nch = (t_end - t_beg + C - 1) / C;
  const int n_last = t_end - t_beg - (nch - 1) * C;          // tokens of the chunk that may be short
  const float g = a.log_decay[h], g2 = g * kLog2e;
  const size_t hs = (size_t)a.K * a.V;
  T* const oh = reinterpret_cast<T*>(a.o) + (size_t)bh * a.T * a.V;

  const HeadRows<T, PK> hk(a.k, a.k_sc, bh, a.T, a.K, t_end);
  const HeadRows<T, PV> hv(a.v, a.v_sc, bh, a.T, a.V, t_end);
  const auto chunk_t0 = [&](int ci) { return t_beg + (REV ? nch - 1 - ci : ci) * C; };
  const auto chunk_n = [&](int ci) { return (REV ? ci == 0 : ci == nch - 1) ? n_last : C; };

  const HeadRows<T, PQ> hq(a.q, a.q_sc, bh, a.T, a.K, t_end);

  // Copies are made by the two output waves that the mask leaves the least to do (a chunk's 24 to 40
  // instructions take the memory pipe 16 cycles each, and a wave that issues them waits): one copies k and half
  // of v, the other q and the rest.  Chunk ci + NS - 1 is requested when chunk ci begins (its place was last read
  // in chunk ci - 1) and has arrived before chunk ci + NS - 2 ends.  8-bit operands pass through registers of
  // all waves: chunk ci + 1 is written to LDS when chunk ci ends, and chunk ci + 2 requested.
  const int issuer = wave >= 4 ? -1 : (NTT == 4 ? (REV ? wave - 2 : wave < 2 ? wave : -1)
                                                : ((wave & 1) == (REV ? 1 : 0) ? wave >> 1 : -1));
  const CopyTile<T, C, KD> ck(lane, a.K, 0);
  const CopyTile<T, C, VT> cv(lane, a.V, v0);
  constexpr int NCK = CopyTile<T, C, KD>::N, NCV = CopyTile<T, C, VT>::N;
  Stage<T, PK, C, KD, NT> pk;
  Stage<T, PV, C, VT, NT> pv;
  Stage<T, PQ, C, KD, NT> pq;
  const auto request = [&](int ci, unsigned at) {
    if (ci < nch) {
      const int t0 = chunk_t0(ci);
      if constexpr (!DMA) {
        pk.load(hk, t0, 0, tid);
        pv.load(hv, t0, v0, tid);
        pq.load(hq, t0, 0, tid);
      } else if (issuer == 0) {
        ck.template issue_range<0, NCK>(hk.words, t0, tile_k(at));
        cv.template issue_range<0, NCV / 2>(hv.words, t0, tile_v(at));
      } else if (issuer == 1) {
        ck.template issue_range<0, NCK>(hq.words, t0, tile_q(at));
        cv.template issue_range<NCV / 2, NCV>(hv.words, t0, tile_v(at));
      }
    }
  };
  const auto stage = [&](int ci, unsigned at) {
    if (ci < nch) {
      pk.store(tile_k(at), tid);
      pv.store(tile_v(at), tid);
      pq.store(tile_q(at), tid);
    }
    request(ci + 1, 0);
  };
  // end of chunk ci: the issuers wait for the next chunk's copies; behind those are the copies of the chunk
  // after it and this wave's stores
  constexpr int COPIES = NCK + NCV / 2, STORES = NO / L::NACC;
  const auto end = [&](int ci, unsigned next) {
    if constexpr (!DMA) {
      stage(ci + 1, next);
    } else if (issuer >= 0) {
      if (NS == 3 && ci + 2 < nch) wait_vm_but<COPIES + STORES>();
      else wait_vm_but<STORES>();
    }
    chunk_barrier();
  };
  request(0, 0);
  if constexpr (DMA && NS == 3) request(1, W::kC);

  unsigned slot = 0;                                           // of chunk ci
  if (wave >= 4) {
    const int rw = wave - 4;
    const int ct0 = rw / W::S::WV * NKS, sv0 = rw % W::S::WV * NVS;
    StateTile<T, KD, VT, C, NKS, NVS, REV> st;
    // (forward: state_out may be state_in, which the last segment may have written before the first one reads)
    const bool first = REV ? t_end == len : a.nseg == 1;
    const float* S0 = !first ? a.seg_state + ((size_t)bh * a.nseg + seg) * hs
                             : (a.state_in ? a.state_in + (size_t)bh * hs : nullptr);
    int mid_seg = REV && a.mid && len > 0 ? (len - 1) / a.midlen : 0;
    if (S0) st.load(S0, a.si_k, a.si_v, ct0, v0 + 16 * sv0, a.K, a.V, lane);
    else st.zero();
    DecaySteps an(g, C);
    const float an_short = decay_pow32(g, nch > 0 ? n_last : 0);
    if (nch > 0) st.image(sS, ct0, 16 * sv0, lane);
    if constexpr (!DMA) stage(0, 0);
    wait_vm_all();
    chunk_barrier();
    for (int ci = 0; ci < nch; ++ci) {
      const int n = chunk_n(ci);
      st.factors(g2, a.u, n, lane);
      const bool fine = fine_state(a.returned, g2, REV ? chunk_t0(ci) : len - chunk_t0(ci) - n);
      st.update(tile_k(slot), tile_v(slot), ct0, sv0, n == C ? an.next() : an_short, fine, lane);
      if constexpr (REV) {
        if (mid_seg > 0 && chunk_t0(ci) == mid_seg * a.midlen) {
          --mid_seg;                             // the states behind this walk's chunks from there on
          int ln = lane;
          asm volatile("" : "+v"(ln));           // (addresses computed here, not kept from before the loop)
          st.save(a.mid + ((size_t)bh * a.nmid + mid_seg) * hs, a.si_k, a.si_v, ct0, v0 + 16 * sv0, a.K, a.V, ln);
        }
      }
      if (ci + 1 < nch) {
        slot = next_slot(slot);
        st.image(sS + (ci + 1 & 1) * W::kS, ct0, 16 * sv0, lane);
        end(ci, slot);
      }
    }
    if (a.state_out && seg == (REV ? 0 : a.nseg - 1))
      st.save(a.state_out + (size_t)bh * hs, a.si_k, a.si_v, ct0, v0 + 16 * sv0, a.K, a.V, lane);
  } else {
    const int ti = wave % NTT, ov0 = wave / NTT * NO;
    const int tl = 16 * ti + (lane & 15);
    const __amdgpu_buffer_rsrc_t ro = make_rsrc(oh, (unsigned)t_end * (unsigned)(a.V * sizeof(T)));
    // c a^{|i - j|} of a score: on the diagonal tile pd (0 where the mask cuts it off), k tiles off it
    // po a^{16 (k - 1)}
    float pd[4], po[4], far[NTT];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int j = 4 * (lane >> 4) + r, d = REV ? j - (lane & 15) : (lane & 15) - j;
      pd[r] = d < 0 ? 0.0f : a.c * decay_pow(g2, d);
      po[r] = a.c * decay_pow(g2, 16 + d);
    }
#pragma unroll
    for (int s = 0; s < NTT; ++s) {
      const int k = REV ? s - ti : ti - s;
      far[s] = k < 1 ? 0.0f : uniform(decay_pow(g2, 16 * (k - 1)));
    }
    if constexpr (!DMA) stage(0, 0);
    wait_vm_all();
    chunk_barrier();
    for (int ci = 0; ci < nch; ++ci) {
      const int n = chunk_n(ci);
      const Lds<T>* cK = tile_k(slot);
      const Lds<T>* cV = tile_v(slot);
      const Lds<T>* cQ = tile_q(slot);
      const Lds<T>* cS = sS + (ci & 1) * W::kS;
      slot = next_slot(slot);
      if constexpr (DMA) request(ci + NS - 1, NS == 3 ? next_slot(slot) : slot);
      frag qf[NQ];
#pragma unroll
      for (int x = 0; x < NQ; ++x) qf[x] = L::template nat<KD, false>(cQ, tl, x * L::DG, lane);
      floatx4 p[L::NACC], acc[NO];
      // scores (keys x tokens) of token group d; the tiles that the mask cuts off come out as zeros.
      // They are rounded to bf16 for the product with V (fp32 walks keep them): one rounding, 2^-8.
      const auto scores = [&](int d) {
#pragma unroll
        for (int s = 0; s < L::NACC; ++s) p[s] = zero4();
        const auto key = [&](int s, int x) {
          return L::template nat<KD, false>(cK, d * L::DG + 16 * s + (lane & 15), x * L::DG, lane);
        };
        // (the outer tile of the diagonal's group may be cut off whole)
        constexpr int IN = REV ? L::NACC - 1 : 0, OUT = L::NACC - 1 - IN;
        const bool outer = REV ? d * L::NACC + OUT >= ti : d * L::NACC + OUT <= ti;
        if (L::NACC == 1 || outer) {
#pragma unroll
          for (int x = 0; x < NQ; ++x)
#pragma unroll
            for (int s = 0; s < L::NACC; ++s) p[s] = L::mma(key(s, x), qf[x], p[s]);
        } else {
#pragma unroll
          for (int x = 0; x < NQ; ++x) p[IN] = L::mma(key(IN, x), qf[x], p[IN]);
        }
#pragma unroll
        for (int s = 0; s < L::NACC; ++s)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int st = d * L::NACC + s;
            p[s][r] *= st == ti ? pd[r] : po[r] * far[st];
          }
        return L::from_acc(p);
      };
      const auto value_out = [&](int d, frag b) {
#pragma unroll
        for (int j = 0; j < NO; ++j) acc[j] = L::mma(L::template tr<VT, true>(cV, ov0 + j, d * L::DG, lane), b, acc[j]);
      };
      // O^T = r a^e S^T Q + V^T scores: token groups 0 and 1 reach this wave's tokens, or only the one
      // that holds them (REV: 1, else 0)
      const bool both = REV ? ti < L::NACC : ti >= L::NACC;
      constexpr int D0 = REV ? 1 : 0, D1 = 1 - D0;
#pragma unroll
      for (int j = 0; j < NO; ++j) acc[j] = zero4();
      const frag p0 = scores(D0);
#pragma unroll
      for (int x = 0; x < NQ; ++x)
#pragma unroll
        for (int j = 0; j < NO; ++j)
          acc[j] = L::mma(L::template nat<KD, true>(cS, L::row_of(ov0 + j, lane & 15), x * L::DG, lane), qf[x], acc[j]);
      const int e = REV ? n - 1 - tl : tl + 1;
      const float rf = a.r * decay_pow(g2, e < 0 ? 0 : e);
#pragma unroll
      for (int j = 0; j < NO; ++j) acc[j] *= rf;
      value_out(D0, p0);
      if (both) value_out(D1, scores(D1));
      const unsigned row = (unsigned)(chunk_t0(ci) + tl) * (unsigned)(a.V * sizeof(T));
#pragma unroll
      for (int j = 0; j < NO; j += L::NACC) {
        const int col = v0 + 16 * (ov0 + j) + (16 / (int)sizeof(T)) * (lane >> 4);
        const unsigned off = col < a.V ? row + (unsigned)(col * sizeof(T)) : 0xfffffff0u;
        __builtin_amdgcn_raw_buffer_store_b128(L::row16(acc + j, lane), ro, off, 0, 0);
      }
      if (ci + 1 < nch) end(ci, slot);
    }
  }
  if (a.zero_tail) {
    const int e_end = (int)min((long long)seg * a.seglen + a.seglen, (long long)a.T);
    const int e_beg = max(len, seg * a.seglen);
    const int w = min(VT, a.V - v0) / L::EPP;                // 16-byte pieces of a row
    for (long long x = tid; x < (long long)(e_end - e_beg) * w; x += NT)
      *reinterpret_cast<u32x4_t*>(oh + (size_t)(e_beg + x / w) * a.V + v0 + (x % w) * L::EPP) = u32x4_t{0, 0, 0, 0};
  }
}

// Workgroups of one walk.
__host__ __device__ inline int walk_blocks(const WalkArgs& a, int VT) { return a.BH * a.nseg * ((a.V + VT - 1) / VT); }

template <typename T, int KD, int VT>
__global__ void __launch_bounds__(kWalkThreads, (WalkShape<T, KD, VT>::EU)) decay_fwd_kernel(WalkArgs a) {
  __shared__ __align__(16) T smem[walk_lds<T, KD, VT, false>()];
  static_assert(sizeof(smem) <= 160 * 1024, "LDS of one gfx950 workgroup exceeded");
  walk<T, KD, VT, false, false, false, false>(a, blockIdx.x, (Lds<T>*)smem);
}

// The three walks of a backward pass in one launch: dq (keys V, values K wide), dk (the same), dv (keys K,
// values V wide).  Each has as many workgroups as the forward has, so that where those fill the chip once
// the other walks' workgroups take the places of the first ones to end, and a small pass costs one launch.
// PACK: q, k and v are kept in 8 bits.  first: the workgroups that an earlier launch had (where dv's segments
// start from states of dk's walk, dv has a launch of its own).
// VT: the widest value tile.
template <typename T, int KD, int VD, bool PACK, int VT> struct BwdShape {
  static constexpr int VTK = KD <= 32 ? 32 : VT, VTV = VD <= 32 ? 32 : VT;        // value tiles over K and over V
  static constexpr int LDS = cmax(walk_lds<T, VD, VTK, PACK>(), walk_lds<T, KD, VTV, PACK>());
  static constexpr int EU = PACK ? 2 : cmin(WalkShape<T, VD, VTK>::EU, WalkShape<T, KD, VTV>::EU);
};
template <typename T, int KD, int VD, bool PACK, int VT>
__global__ void __launch_bounds__(kWalkThreads, (BwdShape<T, KD, VD, PACK, VT>::EU))
    decay_bwd_kernel(WalkArgs dq, WalkArgs dk, WalkArgs dv, int first) {
  typedef BwdShape<T, KD, VD, PACK, VT> S;
  __shared__ __align__(16) T smem[S::LDS];
  static_assert(sizeof(smem) <= 160 * 1024, "LDS of one gfx950 workgroup exceeded");
  const int n = walk_blocks(dq, S::VTK);
  int b = blockIdx.x + first;
  if (b < n) {
    walk<T, VD, S::VTK, false, false, PACK, PACK>(dq, b, (Lds<T>*)smem);
  } else if ((b -= n) < n) {
    walk<T, VD, S::VTK, true, PACK, false, PACK>(dk, b, (Lds<T>*)smem);
  } else {
    walk<T, KD, S::VTV, true, PACK, PACK, false>(dv, b - n, (Lds<T>*)smem);
  }
}

// Chunks in LDS (four or five give the same: it is the state's arithmetic, 1.1 to 1.5 us per chunk, that takes the
// time, 1 x 4 heads of 30011 tokens in 32 segments, K = V = 128, bf16: 22 us; so do tiles of 32 columns).
constexpr int kSegChunks = 3;

// Local end state of one segment (not the last in walking order) for one value tile.
template <typename T, int KD, int VT, int NW, bool REV, bool PK, bool PV>
__device__ __forceinline__ void segment_state(const SegArgs& a, int block, Lds<T>* smem) {
  typedef WalkShape<T, KD, VT> W;
  typedef StateShape<KD, VT, NW> S;
  constexpr int C = W::C, NT = 64 * NW, NS = kSegChunks;
  constexpr bool DMA = !(PK || PV);
  const auto next_slot = [](unsigned s) {
    s = s == (NS - 1) * (W::kK + W::kV) ? 0u : s + (unsigned)(W::kK + W::kV);
    asm volatile("" : "+s"(s));
    return s;
  };
  const int tid = threadIdx.x, lane = tid & 63, sw = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int ntile = (a.V + VT - 1) / VT;
  int idx, tile;
  walk_block(block, a.BH * (a.nseg - 1), ntile, &idx, &tile);
  const int bh = idx / (a.nseg - 1), seg = idx - bh * (a.nseg - 1) + (REV ? 1 : 0), v0 = tile * VT;
  int len = a.T;
  if (a.lengths) len = min(max(a.lengths[bh / a.H], 0), a.T);
  const int t_beg = min(seg * a.seglen, len), t_end = (int)min((long long)seg * a.seglen + a.seglen, (long long)len);
  const int nch = (t_end - t_beg + C - 1) / C;
  const int n_last = t_end - t_beg - (nch - 1) * C;
  const float g = a.log_decay[bh % a.H], g2 = g * kLog2e;
  const HeadRows<T, PK> hk(a.k, a.k_sc, bh, a.T, a.K, t_end);
  const HeadRows<T, PV> hv(a.v, a.v_sc, bh, a.T, a.V, t_end);
  const auto chunk_t0 = [&](int ci) { return t_beg + (REV ? nch - 1 - ci : ci) * C; };
  const auto chunk_n = [&](int ci) { return (REV ? ci == 0 : ci == nch - 1) ? n_last : C; };
  const int ct0 = sw / S::WV * S::NK, sv0 = sw % S::WV * S::NV;
  StateTile<T, KD, VT, C, S::NK, S::NV, REV> st;
  st.zero();
  const Copy<T, C, KD, VT, NW> copy(sw, lane, a.K, a.V, v0);
  Stage<T, PK, C, KD, NT> pk;
  Stage<T, PV, C, VT, NT> pv;
  const auto request = [&](int ci, unsigned at) {
    if (ci < nch) {
      const int t0 = chunk_t0(ci);
      if constexpr (DMA) {
        copy.issue(hk.words, hv.words, t0, a.K, a.V, smem + at, sw);
      } else {
        pk.load(hk, t0, 0, tid);
        pv.load(hv, t0, v0, tid);
      }
    }
  };
  request(0, 0);
  if constexpr (DMA) request(1, W::kK + W::kV);
  unsigned slot = 0;                             // of chunk ci
  DecaySteps an(g, C);
  const float an_short = decay_pow32(g, nch > 0 ? n_last : 0);
  for (int ci = 0; ci < nch; ++ci) {
    const int n = chunk_n(ci);
    if constexpr (DMA) {
      // chunk ci has arrived; the one after it, requested a chunk later, may not have
      if (ci + 1 < nch) wait_vm_but<Copy<T, C, KD, VT, NW>::MIN>();
      else wait_vm_but<0>();
      chunk_barrier();
      request(ci + 2, next_slot(next_slot(slot)));                           // its place was last read in chunk ci - 1
    } else {
      pk.store(smem + slot, tid);
      pv.store(smem + slot + W::kK, tid);
      request(ci + 1, 0);
      chunk_barrier();
    }
    st.factors(g2, a.u, n, lane);
    const bool fine = fine_state(a.returned, g2, REV ? chunk_t0(ci) : len - chunk_t0(ci) - n);
    st.update(smem + slot, smem + slot + W::kK, ct0, sv0, n == C ? an.next() : an_short, fine, lane);
    slot = next_slot(slot);
  }
  st.save(a.seg_state + ((size_t)bh * a.nseg + seg) * a.K * a.V, a.V, 1, ct0, v0 + 16 * sv0, a.K, a.V, lane);
}

// The segments of S (first `nblock` workgroups) and, in a backward pass, those of dL/dS behind them: one
// launch, as either alone may leave half of the chip idle.  PACK: q, k and v are kept in 8 bits.
template <int KD, int VT> constexpr int seg_waves() { return KD == 128 && VT == 64 ? 8 : 4; }
template <typename T, int KD, int VT, bool PACK>
__global__ void __launch_bounds__((64 * seg_waves<KD, VT>())) decay_segment_kernel(SegArgs s, SegArgs r, int nblock) {
  typedef WalkShape<T, KD, VT> W;
  __shared__ __align__(16) T smem[kSegChunks * (W::kK + W::kV)];
  constexpr int NW = seg_waves<KD, VT>();
  if ((int)blockIdx.x < nblock) segment_state<T, KD, VT, NW, false, PACK, PACK>(s, blockIdx.x, (Lds<T>*)smem);
  else segment_state<T, KD, VT, NW, true, PACK, false>(r, blockIdx.x - nblock, (Lds<T>*)smem);
}

// ------------------------------------------------------------------ launchers
// Instances by key and value widths padded to 32, 64 or 128.  Value tiles are 64 columns wide; 32 for widths up
// to 32, and where even those leave every workgroup a CU of its own: then a chunk's time is all that counts, and it
// has half of the products with the state.  (K = V = 128, bf16, 900 tokens, backward: 21 heads 23.6 us in 32
// columns, 30.0 in 64; 22 heads, which pass one round, 38.6 and 30.1; forward 1 x 8 heads 18.4 and 24.5, 64 heads 21.5
// and 26.1, 65 heads 36.2 and 26.0.  fp32, 400 tokens, backward: 21 heads 35.9 and 50.3, 22 heads 65.7 and 50.5.)
constexpr int kNarrowFill = 256;                 // CUs
template <typename T, int KD> hipError_t launch_walk_fwd(const WalkArgs& a, hipStream_t s) {
  if (a.V <= 32 || 2 * walk_blocks(a, 64) <= kNarrowFill)
    hipLaunchKernelGGL((decay_fwd_kernel<T, KD, 32>), dim3(walk_blocks(a, 32)), dim3(kWalkThreads), 0, s, a);
  else
    hipLaunchKernelGGL((decay_fwd_kernel<T, KD, 64>), dim3(walk_blocks(a, 64)), dim3(kWalkThreads), 0, s, a);
  return hipGetLastError();
}

template <typename T, int KD, int VD, bool PACK, int VT>
hipError_t launch_walk_bwd_vt(const WalkArgs& dq, const WalkArgs& dk, const WalkArgs& dv, hipStream_t s) {
  typedef BwdShape<T, KD, VD, PACK, VT> S;
  const int nqk = 2 * walk_blocks(dq, S::VTK), nv = walk_blocks(dv, S::VTV);
  if (!dk.mid) {
    hipLaunchKernelGGL((decay_bwd_kernel<T, KD, VD, PACK, VT>), dim3(nqk + nv), dim3(kWalkThreads), 0, s, dq, dk, dv, 0);
    return hipGetLastError();
  }
  hipLaunchKernelGGL((decay_bwd_kernel<T, KD, VD, PACK, VT>), dim3(nqk), dim3(kWalkThreads), 0, s, dq, dk, dv, 0);
  hipLaunchKernelGGL((decay_bwd_kernel<T, KD, VD, PACK, VT>), dim3(nv), dim3(kWalkThreads), 0, s, dq, dk, dv, nqk);
  return hipGetLastError();
}
template <typename T, int KD, int VD, bool PACK>
hipError_t launch_walk_bwd(const WalkArgs& dq, const WalkArgs& dk, const WalkArgs& dv, hipStream_t s) {
  if constexpr (KD > 32 || VD > 32) {
    if (2 * (2 * walk_blocks(dq, 64) + walk_blocks(dv, 64)) > kNarrowFill)
      return launch_walk_bwd_vt<T, KD, VD, PACK, 64>(dq, dk, dv, s);
  }
  return launch_walk_bwd_vt<T, KD, VD, PACK, 32>(dq, dk, dv, s);
}

template <typename T, int KD, int VT, bool PACK>
hipError_t launch_segments_inst(const SegArgs& st, const SegArgs* r, hipStream_t s) {
  const int blocks = st.BH * (st.nseg - 1) * ((st.V + VT - 1) / VT);
  hipLaunchKernelGGL((decay_segment_kernel<T, KD, VT, PACK>), dim3(r ? 2 * blocks : blocks),
                     dim3(64 * seg_waves<KD, VT>()), 0, s, st, r ? *r : st, blocks);
  return hipGetLastError();
}

// Local states of S (from k, v) and, r non-null, of dL/dS (from q, d_o); packed: q, k, v are in 8 bits.
template <typename T, int KD>
hipError_t launch_segments_kd(const SegArgs& st, const SegArgs* r, bool packed, hipStream_t s) {
  if (st.V <= 32)
    return packed ? launch_segments_inst<T, KD, 32, true>(st, r, s) : launch_segments_inst<T, KD, 32, false>(st, r, s);
  return packed ? launch_segments_inst<T, KD, 64, true>(st, r, s) : launch_segments_inst<T, KD, 64, false>(st, r, s);
}

#define KDA_DECAY_FWD_INSTANCES(EXT, T, KD)                                 \
  EXT template hipError_t launch_walk_fwd<T, KD>(const WalkArgs&, hipStream_t); \
  EXT template hipError_t launch_segments_kd<T, KD>(const SegArgs&, const SegArgs*, bool, hipStream_t);
#define KDA_DECAY_BWD_INSTANCE(EXT, T, KD, VD, PACK) \
  EXT template hipError_t launch_walk_bwd<T, KD, VD, PACK>(const WalkArgs&, const WalkArgs&, const WalkArgs&, hipStream_t);
#define KDA_DECAY_BWD_INSTANCES(EXT, T, KD) \
  KDA_DECAY_BWD_INSTANCE(EXT, T, KD, 32, false) KDA_DECAY_BWD_INSTANCE(EXT, T, KD, 32, true)   \
  KDA_DECAY_BWD_INSTANCE(EXT, T, KD, 64, false) KDA_DECAY_BWD_INSTANCE(EXT, T, KD, 64, true)   \
  KDA_DECAY_BWD_INSTANCE(EXT, T, KD, 128, false) KDA_DECAY_BWD_INSTANCE(EXT, T, KD, 128, true)

}  // namespace kda
