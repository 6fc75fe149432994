// Adjoint of the gated recurrence (kda_gated_scan.h has the mathematics and the way tiles are linked).  Tiles run from
// the last token to the first; r crosses them as the state does forward.  h comes from the kept state in front of the
// tile, so a tile needs its predecessors in one direction only.
#include "kda_gated_scan.h"

#include "../../include/kda.h"

namespace kda {
namespace {

constexpr int S = kScanBwdTokens;

template <int E, int NW> struct ScanShared {
  uint32_t slot;
  float G[NW][E][64], H[NW][E][64], R[NW][E][64], in[E][64];     // sums of g2, states and r from zero
  float2 qg[NW][S][E][64];                 // q and g2 of every token, each lane's own: what the last pass alone needs
};

// The most tokens of any lane's sequence, at least 1.
__device__ __forceinline__ int scan_longest(int n) {
#pragma unroll
  for (int i = 1; i < 64; i *= 2) n = max(n, __shfl_xor(n, i));
  return __builtin_amdgcn_readfirstlane(max(n, 1));
}

// FULL: every token of the tile lies inside its sequence and all channels are their lane's own, in every lane (the same for
// all waves).
template <typename T, int E, int NW, bool GATE, bool NORM, bool GROUPS, bool FULL, typename Off>
__device__ __forceinline__ void scan_bwd_tile(const ScanArgs& a, ScanShared<E, NW>& sh, const ScanTile tile, const ScanLane<E>& l,
                                              int lane, int w) {
  const int jt = a.tiles - 1 - tile.j;     // place in time
  const int t0 = (jt * NW + w) * S;
  const Off row = (Off)a.D * sizeof(T);
  Off base = ((Off)l.bh * a.T + t0) * a.D * sizeof(T) + (Off)l.d * sizeof(T);

  ScanRaw<T, E> rz[S], rx[S], ri[S], rd[S];
#pragma unroll
  for (int k = 0; k < S; ++k) {
    if constexpr (!FULL) rz[k].u = rx[k].u = ri[k].u = rd[k].u = 0;
    if (FULL || t0 + k < l.n) {
      rz[k].load(a.z, base + k * row);
      if constexpr (GATE) ri[k].load(a.i, base + k * row);
      rx[k].load(a.x, base + k * row);
      rd[k].load(a.dy, base + k * row);
    }
  }
  static_assert(NW * S % KDA_GATED_SCAN_CHUNK == 0, "a kept state stands in front of a tile");
  constexpr int per = NW * S / KDA_GATED_SCAN_CHUNK;
  const int chunks = (a.T + KDA_GATED_SCAN_CHUNK - 1) / KDA_GATED_SCAN_CHUNK;
  float h[E];
#pragma unroll
  for (int e = 0; e < E; ++e) h[e] = FULL || jt * NW * S < l.n ? a.ckpt[((size_t)l.bh * chunks + jt * per) * a.D + l.d + e] : 0.f;

  const float m = l.m();
  float bias2[E];
#pragma unroll
  for (int e = 0; e < E; ++e) bias2[e] = l.bias[e] * kLog2e;
  // per token: the decay v, c = n s, sm = 1 - s, k4 = a^2 s x / n; in LDS q = m sigmoid(z') and g2
  float v[S][E], c[S][E], sm[S][E], k4[S][E], G[E], H[E], R[E];
#pragma unroll
  for (int e = 0; e < E; ++e) G[e] = H[e] = R[e] = 0.f;
#pragma unroll
  for (int k = 0; k < S; ++k)
#pragma unroll
    for (int e = 0; e < E; ++e) {
      float y;
      const float p = FULL || t0 + k < l.n ? fmaf(rz[k].at(e), kLog2e, bias2[e]) : kNoDecay;
      const float g = -m * scan_softplus2<true>(p, y);
      sh.qg[w][k][e][lane] = float2{m * fast_rcp(1.f + y) * (p >= 0.f ? 1.f : y), g};
      v[k][e] = decay_of(g);
      const float s = GATE ? scan_sigmoid(ri[k].at(e)) : 1.f, x = rx[k].at(e);
      sm[k][e] = 1.f - s;
      c[k][e] = s;
      k4[k][e] = 0.f;
      if constexpr (NORM) {
        // n = 0 (a decay of exactly 1, or so near it that n^2 is below the normal numbers): the term with 1 / n counts as its
        // limit in dz, 0
        const float n2 = decay_n2(v[k][e]), rn = n2 < 0x1p-126f ? 0.f : __builtin_amdgcn_rsqf(n2), av = 1.f + v[k][e];
        c[k][e] = s * (n2 * rn);
        k4[k][e] = av * av * rn * (s * x);
      }
      G[e] += g;
      H[e] = decay_step(v[k][e], H[e], c[k][e] * x);
      // (kept as they are: what the compiler would compute later from their parts takes more registers)
      asm volatile("" : "+v"(v[k][e]));
      if constexpr (GATE || NORM) asm volatile("" : "+v"(c[k][e]));
      if constexpr (GATE) asm volatile("" : "+v"(sm[k][e]));
      if constexpr (NORM) asm volatile("" : "+v"(k4[k][e]));
    }
#pragma unroll
  for (int k = 0; k < S; ++k) asm volatile("" : "+v"(rx[k].u), "+v"(rd[k].u));
#pragma unroll
  for (int k = S - 1; k >= 0; --k)
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const float r = R[e] + rd[k].at(e);
      R[e] = fmaf(v[k][e], r, r);
    }
#pragma unroll
  for (int e = 0; e < E; ++e) {
    sh.G[w][e][lane] = G[e];
    sh.H[w][e][lane] = H[e];
    sh.R[w][e][lane] = R[e];
  }
  __syncthreads();
  float r[E];
  if (w == 0) {
    // the tiles behind every sequence, which the chain starts after
    const int skip = GROUPS && a.lengths ? a.tiles - (scan_longest(l.n) + NW * S - 1) / (NW * S) : 0;
    const ScanChain chain = scan_chain<E>(a.link, tile.c, a.tiles, skip);
    const bool more = tile.j + 1 < a.tiles;
    float Wt[E], Rt[E];                    // the tile's pair
#pragma unroll
    for (int e = 0; e < E; ++e) Wt[e] = Rt[e] = r[e] = 0.f;
#pragma unroll 1                           // (the registers are full of the wave's tokens)
    for (int p = NW - 1; p >= 0; --p)
#pragma unroll
      for (int e = 0; e < E; ++e) {
        Rt[e] = word_step(word_of(sh.G[p][e][lane]), Rt[e], sh.R[p][e][lane]);
        Wt[e] += sh.G[p][e][lane];
      }
#pragma unroll
    for (int e = 0; e < E; ++e) Wt[e] = word_of(Wt[e]);
    if (!__any(l.n > (jt + 1) * (NW * S))) {     // no sequence goes on behind this tile
      if (a.d_state && l.on)
#pragma unroll
        for (int e = 0; e < E; ++e) r[e] = a.d_state[l.ch + e];
#pragma unroll
      for (int e = 0; e < E; ++e) Rt[e] = word_step(Wt[e], r[e], Rt[e]);
    } else {
      scan_link_tile<E, GROUPS>(chain, tile.j - skip, more, lane, Wt, Rt, r);
    }
#pragma unroll
    for (int e = 0; e < E; ++e) sh.in[e][lane] = r[e];
    if (more) {
      put_words<E>(chain.states + (size_t)(tile.j - skip) * (64 * E) + lane, Rt);
      publish(chain.flags + (tile.j - skip), 2u);
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e)
        if (FULL || l.own(e)) a.d_state_in[l.ch + e] = Rt[e];
    }
  }
  // h in front of this wave's tokens
#pragma unroll 1
  for (int p = 0; p < w; ++p)
#pragma unroll
    for (int e = 0; e < E; ++e) h[e] = word_step(word_of(sh.G[p][e][lane]), h[e], sh.H[p][e][lane]);
  // dg / r = a h_{t-1} - a^2 s x / n of every token
#pragma unroll
  for (int k = 0; k < S; ++k)
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const float ah = fmaf(v[k][e], h[e], h[e]);
      k4[k][e] = ah - k4[k][e];
      h[e] = fmaf(c[k][e], rx[k].at(e), ah);
    }
#pragma unroll
  for (int k = 0; k < S; ++k) asm volatile("" : "+v"(rx[k].u));
  __syncthreads();
  float sz[E], sa[E];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    r[e] = sh.in[e][lane];
    sz[e] = sa[e] = 0.f;
  }
#pragma unroll 1
  for (int p = NW - 1; p > w; --p)
#pragma unroll
    for (int e = 0; e < E; ++e) r[e] = word_step(word_of(sh.G[p][e][lane]), r[e], sh.R[p][e][lane]);
  asm volatile("" : "+v"(base));           // the stores' offsets are computed anew, not kept in registers since the loads
#pragma unroll
  for (int k = S - 1; k >= 0; --k) {
    float dx[E], dz[E], di[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
      r[e] += rd[k].at(e);
      dx[e] = r[e] * c[k][e];
      di[e] = dx[e] * rx[k].at(e) * sm[k][e];
      const float dg = r[e] * k4[k][e];
      const float2 qg = sh.qg[w][k][e][lane];
      dz[e] = -dg * qg.x;
      if (!FULL && t0 + k >= l.n) dx[e] = di[e] = dz[e] = 0.f;
      else {
        sz[e] += dz[e];
        sa[e] = fmaf(dg, qg.y, sa[e]);
      }
      r[e] = fmaf(v[k][e], r[e], r[e]);
    }
    if (FULL || (l.on && t0 + k < a.T)) {
      scan_store<T, E>(a.dx, base + k * row, dx, !FULL && l.last);
      scan_store<T, E>(a.dz, base + k * row, dz, !FULL && l.last);
      if constexpr (GATE) scan_store<T, E>(a.di, base + k * row, di, !FULL && l.last);
    }
  }
  if (!a.parts) return;
  // the waves' sums in a fixed order
#pragma unroll
  for (int e = 0; e < E; ++e) {
    sh.qg[w][0][e][lane] = float2{sz[e], sa[e] * kLn2};        // (in the place of the wave's own, which it has used)
  }
  __syncthreads();
  if (w == 0) {
    const size_t N = (size_t)a.B * a.H * a.D;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      if (!FULL && !l.own(e)) continue;
      float z = 0.f, s = 0.f;
#pragma unroll
      for (int p = 0; p < NW; ++p) {
        const float2 f = sh.qg[p][0][e][lane];
        z += f.x;
        s += f.y;
      }
      a.parts[(size_t)jt * N + l.ch + e] = z;
      a.parts[((size_t)a.tiles + jt) * N + l.ch + e] = s;
    }
  }
}

// A tile behind every lane's sequence: its gradients are zeros.  No other tile waits for it.
template <typename T, int E, int NW, bool GATE, typename Off>
__device__ __forceinline__ void scan_bwd_zeros(const ScanArgs& a, const ScanLane<E>& l, int jt, int w) {
  const float zero[E] = {};
  if (!l.on) return;
  for (int k = 0; k < S; ++k) {
    const int t = (jt * NW + w) * S + k;
    if (t >= a.T) break;
    const Off off = (((Off)l.bh * a.T + t) * a.D + l.d) * sizeof(T);
    scan_store<T, E>(a.dx, off, zero, l.last);
    scan_store<T, E>(a.dz, off, zero, l.last);
    if constexpr (GATE) scan_store<T, E>(a.di, off, zero, l.last);
  }
  if (a.parts && w == 0)
#pragma unroll
    for (int e = 0; e < E; ++e)
      if (l.own(e)) a.parts[(size_t)jt * a.B * a.H * a.D + l.ch + e] = a.parts[((size_t)a.tiles + jt) * a.B * a.H * a.D + l.ch + e] = 0.f;
}

template <typename T, int E, int NW, bool GATE, bool NORM, bool GROUPS, typename Off>
__global__ __launch_bounds__(NW * 64) __attribute__((amdgpu_waves_per_eu(4))) void scan_bwd_kernel(ScanArgs a) {
  __shared__ ScanShared<E, NW> sh;
  const ScanTile tile = scan_tile(a, &sh.slot);
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const ScanLane<E> l = scan_lane<E>(a, tile.c, lane);
  const int jt = a.tiles - 1 - tile.j;
  if (jt > 0 && !__any(l.n > jt * (NW * S))) scan_bwd_zeros<T, E, NW, GATE, Off>(a, l, jt, w);
  else if (__all((jt + 1) * (NW * S) <= l.n && !l.last)) scan_bwd_tile<T, E, NW, GATE, NORM, GROUPS, true, Off>(a, sh, tile, l, lane, w);
  else scan_bwd_tile<T, E, NW, GATE, NORM, GROUPS, false, Off>(a, sh, tile, l, lane, w);
}

template <typename T, int E, int NW, bool GROUPS, typename Off> void launch_nw(const ScanArgs& a, hipStream_t s) {
  const unsigned grid = (unsigned)a.ctiles * (unsigned)a.tiles;
#define KDA_SCAN(G_, N_) scan_bwd_kernel<T, E, NW, G_, N_, GROUPS, Off><<<grid, NW * 64, 0, s>>>(a)
  if (a.i) a.normalize ? KDA_SCAN(true, true) : KDA_SCAN(true, false);
  else a.normalize ? KDA_SCAN(false, true) : KDA_SCAN(false, false);
#undef KDA_SCAN
}
template <typename T, int E, typename Off> void launch_e(const ScanArgs& a, hipStream_t s) {
  if (scan_bwd_waves(a.ctiles) == 4) launch_nw<T, E, 4, false, Off>(a, s);
  else a.link.groups ? launch_nw<T, E, 8, true, Off>(a, s) : launch_nw<T, E, 8, false, Off>(a, s);
}

}  // namespace

template <typename T> hipError_t launch_scan_bwd_tiles(const ScanArgs& a, bool pairs, hipStream_t s) {
  const bool small = (unsigned long long)a.B * a.H * a.T * a.D * sizeof(T) < (1ull << 32);
  if constexpr (sizeof(T) == 2)
    if (pairs) {
      small ? launch_e<T, 2, uint32_t>(a, s) : launch_e<T, 2, size_t>(a, s);
      return hipGetLastError();
    }
  small ? launch_e<T, 1, uint32_t>(a, s) : launch_e<T, 1, size_t>(a, s);
  return hipGetLastError();
}
template hipError_t launch_scan_bwd_tiles<float>(const ScanArgs&, bool, hipStream_t);
template hipError_t launch_scan_bwd_tiles<bf16_t>(const ScanArgs&, bool, hipStream_t);

}  // namespace kda
