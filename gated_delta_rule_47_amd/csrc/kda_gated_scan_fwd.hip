// Forward kernel of the gated recurrence (kda_gated_scan.h has the mathematics and the way tiles are linked).
#include "kda_gated_scan.h"

#include "../../include/kda.h"

namespace kda {
namespace {

constexpr int S = kScanFwdTokens;

template <int E, int NW> struct ScanShared {
  uint32_t slot;
  float G[NW][E][64], W[NW][E][64], H[NW][E][64], in[E][64];     // sums of g2, the decays over them, states from zero
};

// FULL: every token of the tile lies inside its sequence and all channels are their lane's own, in every lane (the same for
// all waves, whose lanes are the same channels).
template <typename T, int E, int NW, bool GATE, bool NORM, bool GROUPS, bool FULL, typename Off>
__device__ __forceinline__ void scan_fwd_tile(const ScanArgs& a, ScanShared<E, NW>& sh, const ScanTile tile, const ScanLane<E>& l,
                                              int lane, int w) {
  const int t0 = (tile.j * NW + w) * S;
  const Off row = (Off)a.D * sizeof(T);
  Off base = ((Off)l.bh * a.T + t0) * a.D * sizeof(T) + (Off)l.d * sizeof(T);

  ScanRaw<T, E> rz[S], rx[S], ri[S];
#pragma unroll
  for (int k = 0; k < S; ++k) {
    if constexpr (!FULL) rz[k].u = rx[k].u = ri[k].u = 0;
    if (FULL || t0 + k < l.n) {
      rz[k].load(a.z, base + k * row);
      rx[k].load(a.x, base + k * row);
      if constexpr (GATE) ri[k].load(a.i, base + k * row);
    }
  }
  const float m = l.m();
  float bias2[E];
#pragma unroll
  for (int e = 0; e < E; ++e) bias2[e] = l.bias[e] * kLog2e;
  float v[S][E], u[S][E], G[E], H[E];
#pragma unroll
  for (int e = 0; e < E; ++e) G[e] = H[e] = 0.f;
#pragma unroll
  for (int k = 0; k < S; ++k)
#pragma unroll
    for (int e = 0; e < E; ++e) {
      float y;
      const float p = FULL || t0 + k < l.n ? fmaf(rz[k].at(e), kLog2e, bias2[e]) : kNoDecay;
      const float g2 = -m * scan_softplus2(p, y);
      float uu = rx[k].at(e);
      if constexpr (GATE) uu *= scan_sigmoid(ri[k].at(e));
      const float d = decay_of(g2);
      if constexpr (NORM) uu *= __builtin_amdgcn_sqrtf(decay_n2(d));
      v[k][e] = d;
      u[k][e] = uu;
      G[e] += g2;
      H[e] = decay_step(d, H[e], uu);
      asm volatile("" : "+v"(v[k][e]), "+v"(u[k][e]));     // (not to be computed later from parts that take more registers)
    }
#pragma unroll
  for (int e = 0; e < E; ++e) {
    sh.G[w][e][lane] = G[e];
    sh.W[w][e][lane] = word_of(G[e]);
    sh.H[w][e][lane] = H[e];
  }
  __syncthreads();
  float h[E];
  if (w == NW - 1) {
    const ScanChain chain = scan_chain<E>(a.link, tile.c, a.tiles, 0);
    const bool more = tile.j + 1 < a.tiles;
    float Wt[E], Ht[E];                    // the tile's pair
#pragma unroll
    for (int e = 0; e < E; ++e) Wt[e] = Ht[e] = h[e] = 0.f;
#pragma unroll 1                           // (the registers are full of the wave's tokens)
    for (int p = 0; p < NW; ++p)
#pragma unroll
      for (int e = 0; e < E; ++e) {
        Ht[e] = word_step(sh.W[p][e][lane], Ht[e], sh.H[p][e][lane]);
        Wt[e] += sh.G[p][e][lane];
      }
#pragma unroll
    for (int e = 0; e < E; ++e) Wt[e] = word_of(Wt[e]);
    if (tile.j == 0) {
      if (a.state_in)                      // (another lane's channel may have its last state there by now)
#pragma unroll
        for (int e = 0; e < E; ++e) h[e] = FULL || l.own(e) ? a.state_in[l.ch + e] : 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) Ht[e] = word_step(Wt[e], h[e], Ht[e]);
    } else {
      scan_link_tile<E, GROUPS>(chain, tile.j, more, lane, Wt, Ht, h);
    }
#pragma unroll
    for (int e = 0; e < E; ++e) sh.in[e][lane] = h[e];
    if (more) {
      put_words<E>(chain.states + (size_t)tile.j * (64 * E) + lane, Ht);
      publish(chain.flags + tile.j, 2u);
    }
  }
  __syncthreads();
#pragma unroll
  for (int e = 0; e < E; ++e) h[e] = sh.in[e][lane];
#pragma unroll 1
  for (int p = 0; p < w; ++p)
#pragma unroll
    for (int e = 0; e < E; ++e) h[e] = word_step(sh.W[p][e][lane], h[e], sh.H[p][e][lane]);
  static_assert(KDA_GATED_SCAN_CHUNK % S == 0, "a kept state stands in front of a wave's tokens");
  if (a.ckpt && t0 % KDA_GATED_SCAN_CHUNK == 0 && t0 < l.n) {
    const int chunks = (a.T + KDA_GATED_SCAN_CHUNK - 1) / KDA_GATED_SCAN_CHUNK;
#pragma unroll
    for (int e = 0; e < E; ++e)
      if (FULL || l.own(e)) a.ckpt[((size_t)l.bh * chunks + t0 / KDA_GATED_SCAN_CHUNK) * a.D + l.d + e] = h[e];
  }
  asm volatile("" : "+v"(base));           // the stores' offsets are computed anew, not kept in registers since the loads
#pragma unroll
  for (int k = 0; k < S; ++k) {
#pragma unroll
    for (int e = 0; e < E; ++e) h[e] = decay_step(v[k][e], h[e], u[k][e]);
    if (FULL || t0 + k < l.n) scan_store<T, E>(a.y, base + k * row, h, !FULL && l.last);
  }
  // the tile of a sequence's last token (or the first one) has its final state: behind it the state stays
  const int start = tile.j * (NW * S);
  if (w == NW - 1 && a.state_out && l.n <= start + NW * S && (l.n > start || tile.j == 0))
#pragma unroll
    for (int e = 0; e < E; ++e)
      if (FULL || l.own(e)) a.state_out[l.ch + e] = h[e];
}

template <typename T, int E, int NW, bool GATE, bool NORM, bool GROUPS, typename Off>
__global__ __launch_bounds__(NW * 64) __attribute__((amdgpu_waves_per_eu(4))) void scan_fwd_kernel(ScanArgs a) {
  __shared__ ScanShared<E, NW> sh;
  const ScanTile tile = scan_tile(a, &sh.slot);
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const ScanLane<E> l = scan_lane<E>(a, tile.c, lane);
  if (tile.j > 0 && !__any(l.n > tile.j * (NW * S))) return;     // behind every lane's sequence, as are the tiles after it
  if (__all((tile.j + 1) * (NW * S) <= l.n && !l.last)) scan_fwd_tile<T, E, NW, GATE, NORM, GROUPS, true, Off>(a, sh, tile, l, lane, w);
  else scan_fwd_tile<T, E, NW, GATE, NORM, GROUPS, false, Off>(a, sh, tile, l, lane, w);
}

template <typename T, int E, int NW, bool GROUPS, typename Off> void launch_nw(const ScanArgs& a, hipStream_t s) {
  const unsigned grid = (unsigned)a.ctiles * (unsigned)a.tiles;
#define KDA_SCAN(G_, N_) scan_fwd_kernel<T, E, NW, G_, N_, GROUPS, Off><<<grid, NW * 64, 0, s>>>(a)
  if (a.i) a.normalize ? KDA_SCAN(true, true) : KDA_SCAN(true, false);
  else a.normalize ? KDA_SCAN(false, true) : KDA_SCAN(false, false);
#undef KDA_SCAN
}
template <typename T, int E, typename Off> void launch_e(const ScanArgs& a, hipStream_t s) {
  if (scan_fwd_waves(a.ctiles) == 4) launch_nw<T, E, 4, false, Off>(a, s);
  else a.link.groups ? launch_nw<T, E, 8, true, Off>(a, s) : launch_nw<T, E, 8, false, Off>(a, s);
}

}  // namespace

template <typename T> hipError_t launch_scan_fwd_tiles(const ScanArgs& a, bool pairs, hipStream_t s) {
  const bool small = (unsigned long long)a.B * a.H * a.T * a.D * sizeof(T) < (1ull << 32);
  if constexpr (sizeof(T) == 2)
    if (pairs) {
      small ? launch_e<T, 2, uint32_t>(a, s) : launch_e<T, 2, size_t>(a, s);
      return hipGetLastError();
    }
  small ? launch_e<T, 1, uint32_t>(a, s) : launch_e<T, 1, size_t>(a, s);
  return hipGetLastError();
}
template hipError_t launch_scan_fwd_tiles<float>(const ScanArgs&, bool, hipStream_t);
template hipError_t launch_scan_fwd_tiles<bf16_t>(const ScanArgs&, bool, hipStream_t);

}  // namespace kda
