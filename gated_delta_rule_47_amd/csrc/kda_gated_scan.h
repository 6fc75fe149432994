// Gated linear recurrence, one state per channel: what the forward, the adjoint and the single token share.
//
//   g = -m softplus(z + dt_bias), m = exp(clamp(A_log, -10, 20)),  a = e^g,  n = (1 - a^2)^1/2 or 1,  s = sigmoid(i) or 1
//   h_t = a_t h_{t-1} + n_t s_t x_t,  y = h
//   r_t = dL/dh_t = dy_t + a_{t+1} r_{t+1}:  dx = r n s,  di = r n x s (1 - s),
//   dg = r (a h_{t-1} - a^2 / n s x),  dz = -dg m sigmoid(z + dt_bias),  dA_log = sum dg g,  ddt_bias = sum dz
//
// Channels of all heads and sequences stand side by side, E neighbours of one head to a lane (E = 2 packs a 4-byte
// access of bf16; fp32 takes 1), 64 lanes to a channel tile.  The last lane of an odd head has the channel in front of its
// own too, computes it as its neighbour does and stores nothing of it (training step of 4 x 8192 x 2049, bf16: 432 us, 481
// with one channel a lane).  Time is cut into tiles of NW waves of S tokens, one workgroup each.  A wave keeps the decays
// and inputs of its S tokens in registers, so memory is read once: it folds them to one pair (decay over all of them,
// state from zero), the workgroup's waves put these into LDS, one wave fetches the state in front of the tile from the
// tiles before it (scan_link_tile); then every wave takes that state over the pairs of the waves in front of it and runs over
// its tokens again from the true one.
//
// Tiles hand their states on through the workspace.  Each publishes its own pair as soon as it has it, without
// waiting for anything, then takes the pairs of the tiles before it from the nearest one on that knows its final state,
// and publishes its own final state.  A channel tile's workgroups take its tiles by a counter, in time order: whatever a
// tile waits for belongs to a workgroup that already runs, and a pair is published without waiting (a group's pair waits
// for its tiles' pairs alone), so every wait ends.  (One counter per channel tile, on a line of its own: with a single one
// the padded batch of 8 x 8 x 4096 x 64 took 48 us for 42.)  Words are written and read by device-scope atomics (past the
// XCDs' own L2), each record complete before its flag.
//
// Bound by memory and next to it by the vector unit (about 52 and 69 instructions an element, transcendentals among them, busy
// 60 to 70 % of the time).  Measured, bf16 with both gates: forward, 8 x 8192 x 4096, 434 us (4.95 TB/s), 1 x 30011 x 4096, 222 us
// (4.4); adjoint, 4 x 8192 x 2048, 214 us (4.4); one token of 192 x 4096, 4.6 us.
#pragma once

#include "kda_launch.h"
#include "kda_vec.h"

namespace kda {

__device__ __forceinline__ float scan_sigmoid(float x) { return fast_rcp(1.0f + fast_exp2(-kLog2e * x)); }

// log2(1 + 2^x2) for every x2 >= 0 or below: with y = 2^-|x2| and u = fl(1 + y), log2(1 + y) = log2(u) + (y - (u - 1)) / u
// log2(e) + ..., and the correction only matters where u is next to 1 (y itself where u rounds to 1).
// FINITE holds it at 1e20, where any multiplier (e^-10 to e^20) gives a decay of 0 and a finite g2: in the multiplier's gradient
// dg g2 is then 0, as the limit is, not 0 times infinity (a NaN stays one through y).  The adjoint alone needs that; the
// forward pass gives the same bits without it, and took 1 % longer with it (1 x 30011 x 4096).
template <bool FINITE = false> __device__ __forceinline__ float scan_softplus2(float x2, float& y) {
  y = fast_exp2(-fabsf(x2));
  const float u = 1.0f + y;
  return fmaf(y - (u - 1.0f), kLog2e, fast_log2(u)) + (FINITE ? __builtin_amdgcn_fmed3f(x2, 0.f, 1e20f) : fmaxf(x2, 0.f));
}

// A token's decay e^g, g = g2 ln 2 <= 0, is held as e = e^g - 1.  A decay next to 1 rounded to fp32 would be off to the same
// side in every token of a channel whose gate hardly moves, by up to 2^-25 / |g| of the state after the 1 / |g| tokens it
// remembers; e is right to a rounding of itself there.  (Next to 0 it is right to 2^-25: what is left of a state after a
// strong decay is right to 2^-24 of what it was a token before.)  For |g| < 1/8, e / g2 is a cubic within 3.5e-8 of
// (2^g2 - 1) / g2 (interpolated at Chebyshev points).
constexpr float kWeak = -0.18033688f;      // -1/8 in units of log2(e)
__device__ __forceinline__ float decay_weak(float g2) {
  return g2 * fmaf(g2, fmaf(g2, fmaf(g2, 0.009150667116f, 0.05545188114f), 0.2402246296f), 0.6931471825f);
}
__device__ __forceinline__ float decay_of(float g2) {
  const float e = decay_weak(g2), f = fast_exp2(g2) - 1.0f;          // (both, and a selection: no branch)
  return g2 > kWeak ? e : f;
}
__device__ __forceinline__ float decay_step(float e, float h, float u) { return fmaf(e, h, h) + u; }   // a h + u
__device__ __forceinline__ float decay_n2(float e) { return -e * (2.f + e); }                         // 1 - a^2

// The decay over many tokens in one word, which keeps its relative accuracy at both ends (a state may have been larger
// than what is left of it by any factor): next to 1 its distance from 1, with the sign bit set even for 0, the decay
// itself otherwise.
__device__ __forceinline__ bool word_weak(float w) { return (int)__float_as_uint(w) < 0; }
__device__ __forceinline__ float word_of(float g2) {
  const float e = -fabsf(decay_weak(g2)), a = fast_exp2(g2);
  return g2 > kWeak ? e : a;
}
// The decay over both: two distances from 1 as long as theirs is below a half.
__device__ __forceinline__ float word_join(float v, float w) {
  const bool x = word_weak(v), y = word_weak(w);
  const float e = fmaf(v, w, v) + w, a = (x ? 1.f + v : v) * (y ? 1.f + w : w);
  return x && y && e > -0.5f ? -fabsf(e) : a;
}
__device__ __forceinline__ float word_step(float w, float h, float u) { return fmaf(w, h, (word_weak(w) ? h : 0.f) + u); }

// A gate's argument (in units of log2(e)) whose softplus is 0, for tokens behind a sequence: g = 0, the state stays, and
// with inputs of 0 nothing is added to it.
constexpr float kNoDecay = -1e30f;

// E elements of a row as loaded, at a byte offset from the tensor's start (32 bits where the tensors are below 4 GiB:
// one offset then serves every tensor, which stay in scalar registers).
template <typename T, int E> struct ScanRaw {
  uint32_t u;
  static_assert((int)sizeof(T) * E <= 4, "one word");
  template <typename Off> __device__ __forceinline__ void load(const void* p, Off off) {
    const char* q = (const char*)p + off;
    if constexpr (sizeof(T) * E == 4) u = reinterpret_cast<const Words<1, sizeof(T)>*>(q)->u[0];
    else u = *reinterpret_cast<const uint16_t*>(q);
  }
  __device__ __forceinline__ float at(int e) const {
    if constexpr (sizeof(T) == 4) return __uint_as_float(u);
    else return __uint_as_float(e ? u & 0xffff0000u : u << 16);
  }
};
template <typename T, int E, typename Off> __device__ __forceinline__ void scan_store(void* p, Off off, const float (&f)[E]) {
  char* q = (char*)p + off;
  if constexpr (sizeof(T) == 4) *reinterpret_cast<float*>(q) = f[0];
  else if constexpr (E == 2) reinterpret_cast<Words<1, sizeof(T)>*>(q)->u[0] = pack_bf16x2(f[0], f[1]);
  else *reinterpret_cast<bf16_t*>(q) = f2bf(f[0]);
}
// `last`: the last element alone.
template <typename T, int E, typename Off> __device__ __forceinline__ void scan_store(void* p, Off off, const float (&f)[E], bool last) {
  if constexpr (E == 2)
    if (last) {
      scan_store<T, 1>(p, off + (Off)sizeof(T), {f[1]});
      return;
    }
  scan_store<T, E>(p, off, f);
}

// What links the tiles of a channel tile: a counter (every `every` words), a flag per tile (0 nothing, 1 its pair, 2 its final
// state too), the records (64 lanes of E pairs, 64 lanes of E states); a flag (1: its pair) and a pair per group of tiles.
struct ScanLink {
  uint32_t *tickets, *flags, *group_flags;
  uint32_t every, groups;                  // groups of a channel tile, 0: none
  float *pairs, *states, *group_pairs;
};
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
  float *d_state_in, *parts;               // (2, tiles, B H D): sums of dz, of dg g
  ScanLink link;
  int B, H, T, D, normalize, ctiles, tiles;
};

// A lane's E floats by device-scope accesses.
template <int E> __device__ __forceinline__ void put_words(float* p, const float (&f)[E]) {
#pragma unroll
  for (int e = 0; e < E; ++e) __hip_atomic_store(p + e * 64, f[e], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
template <int E> __device__ __forceinline__ void get_words(const float* p, float (&f)[E]) {
#pragma unroll
  for (int e = 0; e < E; ++e) f[e] = __hip_atomic_load(p + e * 64, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
// The record's stores have reached memory before the flag is written.
__device__ __forceinline__ void publish(uint32_t* flag, uint32_t value) {
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  if ((threadIdx.x & 63) == 0) __hip_atomic_store(flag, value, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// The flags of 64 places, from place `at` (bit 0) towards the first: which have one (1 or 2), which have 2.
struct ScanFlags {
  unsigned long long any, final;
};
// The nearest place p <= last with flag 2 where all places behind it have theirs (1 or 2).  A place without
// one belongs to a workgroup that runs and will publish; nearer places may have finished since, so it starts again.
// (Without a GPU in it: read(at) gives the flags of a window, pause() waits a little.)
template <typename Read, typename Pause> __host__ __device__ __forceinline__ int scan_look_back(int last, Read read, Pause pause) {
  for (int at = last;;) {                  // the newest place of a window of 64
    const ScanFlags f = read(at);
    const unsigned long long none = ~f.any;
    const int ready = none ? __builtin_ctzll(none) : 64, stop = f.final ? __builtin_ctzll(f.final) : 64;
    if (stop < ready) return at - stop;
    if (ready == 64) {
      at -= 64;
    } else {
      at = last;
      pause();
    }
  }
}
// The same over flag(p), by one wave.
template <typename Flag> __device__ __forceinline__ int scan_nearest(int last, int lane, Flag flag) {
  return scan_look_back(
      last,
      [&](int at) {
        const uint32_t f = flag(at - lane);
        return ScanFlags{__ballot(f >= 1u), __ballot(f == 2u)};
      },
      [] { __builtin_amdgcn_s_sleep(1); });
}
__device__ __forceinline__ uint32_t scan_flag(const uint32_t* p) {
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
// h taken over the pairs of places k0 .. k1 - 1; with W also the decay over them.
template <int E, bool WORDS> __device__ __forceinline__ void scan_fold(const float* pairs, int k0, int k1, int lane, float (&h)[E],
                                                                      float (&W)[E]) {
  constexpr int U = 2;
#pragma unroll 1
  for (int k = k0; k < k1; k += U) {
    float pg[U][E], ph[U][E];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const float* r = pairs + (size_t)min(k + u, k1 - 1) * (128 * E) + lane;
      get_words<E>(r, pg[u]);
      get_words<E>(r + 64 * E, ph[u]);
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (k + u < k1)
#pragma unroll
        for (int e = 0; e < E; ++e) {
          h[e] = word_step(pg[u][e], h[e], ph[u][e]);
          if constexpr (WORDS) W[e] = word_join(W[e], pg[u][e]);
        }
  }
}

// Tiles of a group: 2^kScanGroupLog2, up to 64.  Few channels over a long time put hundreds of tiles to work at once, which
// wait for joins one behind the other (0.2 us each); with groups a tile is as many joins away from a known state as there
// are groups in front of it and tiles in its own.  1 x 32768 x 64, bf16, forward and adjoint: 25 and 54 us, 55 and 114 without.
constexpr int kScanGroupLog2 = 3;
// Where a tile's predecessors have mostly finished, a group's pair is one more wait: 1 x 16384 x 2048 (16 channel tiles),
// 79 and 155 us with groups, 69 and 138 without; 8 channel tiles (1 x 8192 x 1024), 28 and 52 both ways.  Up to 32 tiles the
// two are alike (1 x 4096 x 512 forward: 17.0 us).
constexpr bool scan_grouped(int ctiles, int tiles) { return ctiles <= 8 && tiles > 32; }

// The links of one channel tile, from its first tile that has tokens on.
struct ScanChain {
  uint32_t *flags, *group_flags;
  float *pairs, *states, *group_pairs;
};
template <int E> __device__ __forceinline__ ScanChain scan_chain(const ScanLink& l, int c, int tiles, int skip) {
  const size_t first = (size_t)c * tiles + skip, g = (size_t)c * l.groups;
  return {l.flags + first, l.group_flags + g, l.pairs + first * (128 * E), l.states + first * (64 * E),
          l.group_pairs + g * (128 * E)};
}
// State in front of group k > 0: from the nearest group whose last tile knows its final state, over the groups' pairs.
template <int E> __device__ __forceinline__ void scan_group_start(const ScanChain& c, int k, int lane, float (&h)[E]) {
  constexpr int shift = kScanGroupLog2;
  const int from = scan_nearest(k - 1, lane, [&](int q) {
    if (q < 0) return 0u;
    if (scan_flag(c.flags + ((q + 1) << shift) - 1) == 2u) return 2u;
    return q ? scan_flag(c.group_flags + q) : 0u;
  });
  asm volatile("" ::: "memory");
  get_words<E>(c.states + (size_t)(((from + 1) << shift) - 1) * (64 * E) + lane, h);
  scan_fold<E, false>(c.group_pairs, from + 1, k, lane, h, h);
}
// Tile j > 0 of a chain, one wave: publishes its pair (W, H), gives the state h in front of it and in H its final one.
// It starts from the nearest tile that knows its final state and takes the pairs behind it one after the other, as each of
// those tiles does for its own final state: so the result is the same bit by bit wherever it starts.
// With groups this ends at the group's first tile, and the state in front of a group comes from the groups in front of
// it in the same way: the last tile of a group joins its pairs to one, and its final state is by definition the state in
// front of the group taken over that.  (Group 0 has no pair: its last tile's state is taken over its tiles.)
template <int E, bool GROUPS>
__device__ __forceinline__ void scan_link_tile(const ScanChain& c, int j, bool more, int lane, float (&W)[E], float (&H)[E],
                                               float (&h)[E]) {
  constexpr int shift = GROUPS ? kScanGroupLog2 : 31;
  float* pair = c.pairs + (size_t)j * (128 * E) + lane;
  put_words<E>(pair, W);
  put_words<E>(pair + 64 * E, H);
  publish(c.flags + j, 1u);
  const int k = j >> shift, j0 = k << shift;
  const bool closes = GROUPS && k > 0 && more && (j + 1) >> shift > k;
  int from = j0 - 1;
  if (closes) {
    while (__any(lane < j - j0 && scan_flag(c.flags + j0 + lane) == 0u)) __builtin_amdgcn_s_sleep(1);
    asm volatile("" ::: "memory");
    float Wg[E], Hg[E];
#pragma unroll
    for (int e = 0; e < E; ++e) Wg[e] = -0.f, Hg[e] = 0.f;
    scan_fold<E, true>(c.pairs, j0, j, lane, Hg, Wg);
#pragma unroll
    for (int e = 0; e < E; ++e) {
      H[e] = word_step(W[e], Hg[e], H[e]);
      W[e] = word_join(Wg[e], W[e]);
    }
    float* gp = c.group_pairs + (size_t)k * (128 * E) + lane;
    put_words<E>(gp, W);
    put_words<E>(gp + 64 * E, H);
    publish(c.group_flags + k, 1u);
  } else {
    from = scan_nearest(j - 1, lane, [&](int p) { return p >= j0 ? scan_flag(c.flags + p) : k ? 2u : 0u; });
    asm volatile("" ::: "memory");
  }
  if (!GROUPS || from >= j0) get_words<E>(c.states + (size_t)from * (64 * E) + lane, h);
  else scan_group_start<E>(c, k, lane, h);
#pragma unroll
  for (int e = 0; e < E; ++e)
    if (closes) H[e] = word_step(W[e], h[e], H[e]);
  scan_fold<E, false>(c.pairs, from + 1, j, lane, h, h);
#pragma unroll
  for (int e = 0; e < E; ++e)
    if (!closes) H[e] = word_step(W[e], h[e], H[e]);
}

// The tile of this workgroup: channel tile c, place j in the order of the tickets.
struct ScanTile {
  int c, j;
};
__device__ __forceinline__ ScanTile scan_tile(const ScanArgs& a, uint32_t* slot) {
  const uint32_t c = blockIdx.x % (uint32_t)a.ctiles;
  uint32_t j = 0;
  if (a.tiles > 1) {
    if (threadIdx.x == 0)
      *slot = __hip_atomic_fetch_add(a.link.tickets + c * a.link.every, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    __syncthreads();
    j = (uint32_t)__builtin_amdgcn_readfirstlane((int)*slot);
  }
  return {(int)c, (int)j};
}

// A lane's channels: index among all of them, head, sequence's tokens, parameters.
template <int E> struct ScanLane {
  long long ch;
  int h, d, n;
  long long bh;
  bool on, last;                           // last: only the last of the E channels is this lane's own
  __device__ __forceinline__ bool own(int e) const { return on && (e == E - 1 || !last); }
  float a_log, bias[E];                    // as loaded: nothing waits for them before the tile's own loads are issued
  __device__ __forceinline__ float m() const { return gate_multiplier(a_log); }
};
template <int E> __device__ __forceinline__ ScanLane<E> scan_lane(const ScanArgs& a, int c, int lane) {
  const uint32_t per = (uint32_t)(a.D + E - 1) / E, at = (uint32_t)c * 64 + (uint32_t)lane;      // B H D <= 2^26
  ScanLane<E> l;
  l.on = at < (uint32_t)(a.B * a.H) * per;
  const uint32_t bh = l.on ? at / per : 0u;
  l.bh = bh;
  l.d = l.on ? (int)(at - bh * per) * E : 0;
  l.last = l.d + E > a.D;
  if (l.last) l.d = a.D - E;
  l.ch = l.bh * a.D + l.d;
  const uint32_t b = bh / (uint32_t)a.H;
  l.h = (int)(bh - b * (uint32_t)a.H);
  l.n = !l.on ? 0 : a.lengths ? min(max(a.lengths[b], 0), a.T) : a.T;
  l.a_log = a.A_log[l.h];
#pragma unroll
  for (int e = 0; e < E; ++e) l.bias[e] = 0.f;
  if (a.dt_bias)
#pragma unroll
    for (int e = 0; e < E; ++e) l.bias[e] = a.dt_bias[(size_t)l.h * a.D + l.d + e];
  return l;
}

// Tile shapes.  Forward: S = 16 tokens of decay and input are 64 registers at E = 2; eight waves, or four where the channel
// tiles are many (scan_fwd_waves).  Backward: four values a token in registers and two in LDS.
constexpr int kScanFwdTokens = 16, kScanBwdTokens = 8;
// Five workgroups of four waves fit a CU and two of eight.  The smaller ones overlap better (8 x 8192 x 4096: 434 us for 460) and
// put twice as many tiles into a channel's line, of which 256 CUs hold more at once the fewer channels there are (1 x
// 30011 x 4096: 241 us for 222).
constexpr int scan_fwd_waves(int ctiles) { return ctiles >= 128 ? 4 : 8; }
// Backward, four workgroups of four waves fit a CU or two of eight, which halve a channel's line of tiles: 1 x 16384 x 4096,
// 239 us for 264, 2 x 8 x 32768 x 64 in fp32, 268 for 333; from 64 channel tiles on the line is short enough (1 x 4096 x 8192: 126 us for 124).
constexpr int scan_bwd_waves(int ctiles) { return ctiles >= 64 ? 4 : 8; }

template <typename T> hipError_t launch_scan_fwd_tiles(const ScanArgs& a, bool pairs, hipStream_t s);
template <typename T> hipError_t launch_scan_bwd_tiles(const ScanArgs& a, bool pairs, hipStream_t s);

}  // namespace kda
