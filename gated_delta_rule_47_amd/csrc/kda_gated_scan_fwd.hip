// Forward kernel of the gated recurrence (kda_gated_scan.h has the mathematics and the way tiles are linked).
#include "kda_gated_scan.h"

#include "../../include/kda.h"

namespace kda {
namespace {

constexpr int NW = kScanFwdWaves, S = kScanFwdTokens;

template <typename T, int E, bool GATE, bool NORM, typename Off>
__global__ __launch_bounds__(NW * 64) __attribute__((amdgpu_waves_per_eu(4))) void scan_fwd_kernel(ScanArgs a) {
  __shared__ uint32_t slot;
  __shared__ float sG[NW][E][64], sH[NW][E][64], sIn[E][64];
  const ScanTile tile = scan_tile(a, &slot);
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const ScanLane<E> l = scan_lane<E>(a, tile.c, lane);
  const int t0 = (tile.j * NW + w) * S;
  const Off row = (Off)a.D * sizeof(T);
  const Off base = ((Off)l.bh * a.T + t0) * a.D * sizeof(T) + (Off)l.d * sizeof(T);
  const bool full = __all(t0 + S <= l.n);

  ScanRaw<T, E> rz[S], rx[S], ri[S];
  if (full) {
#pragma unroll
    for (int k = 0; k < S; ++k) {
      rz[k].load(a.z, base + k * row);
      rx[k].load(a.x, base + k * row);
      if constexpr (GATE) ri[k].load(a.i, base + k * row);
    }
  } else {
#pragma unroll
    for (int k = 0; k < S; ++k) {
      rz[k].u = rx[k].u = ri[k].u = 0;
      if (t0 + k < l.n) {
        rz[k].load(a.z, base + k * row);
        rx[k].load(a.x, base + k * row);
        if constexpr (GATE) ri[k].load(a.i, base + k * row);
      }
    }
  }
  float v[S][E], u[S][E], G[E], H[E];
#pragma unroll
  for (int e = 0; e < E; ++e) G[e] = H[e] = 0.f;
#pragma unroll
  for (int k = 0; k < S; ++k)
#pragma unroll
    for (int e = 0; e < E; ++e) {
      float y;
      float g2 = -l.m * scan_softplus2(fmaf(rz[k].at(e), kLog2e, l.bias2[e]), y);
      float uu = rx[k].at(e);
      v[k][e] = decay_word(g2);
      if constexpr (GATE) uu *= scan_sigmoid(ri[k].at(e));
      if constexpr (NORM) uu *= __builtin_amdgcn_sqrtf(decay_n2(v[k][e]));
      if (!full && t0 + k >= l.n) {        // behind the sequence: the state stays
        v[k][e] = kNoDecay;
        uu = g2 = 0.f;
      }
      u[k][e] = uu;
      G[e] += g2;
      H[e] = decay_step(v[k][e], H[e], uu);
    }
#pragma unroll
  for (int e = 0; e < E; ++e) {
    sG[w][e][lane] = G[e];
    sH[w][e][lane] = H[e];
  }
  __syncthreads();
  // the waves in front of this one, from a state of zero
  float Gp[E], Hp[E];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    Gp[e] = Hp[e] = 0.f;
    for (int p = 0; p < w; ++p) {
      Hp[e] = decay_step(decay_word(sG[p][e][lane]), Hp[e], sH[p][e][lane]);
      Gp[e] += sG[p][e][lane];
    }
  }
  if (w == NW - 1) {
    float Gt[E], Ht[E], in[E];
    const size_t first = (size_t)tile.c * a.tiles, rec = first + tile.j;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      Ht[e] = decay_step(decay_word(G[e]), Hp[e], H[e]);
      Gt[e] = Gp[e] + G[e];
      in[e] = 0.f;
    }
    if (tile.j == 0) {
      if (a.state_in && l.on)
#pragma unroll
        for (int e = 0; e < E; ++e) in[e] = a.state_in[l.ch + e];
    } else {
      float* pair = a.link.pairs + rec * (128 * E) + lane;
      put_words<E>(pair, Gt);
      put_words<E>(pair + 64 * E, Ht);
      publish(a.link.flags + rec, 1u);
      look_back<E>(a.link, first, tile.j, lane, in);
    }
#pragma unroll
    for (int e = 0; e < E; ++e) {
      sIn[e][lane] = in[e];
      Ht[e] = decay_step(decay_word(Gt[e]), in[e], Ht[e]);
    }
    if (tile.j + 1 < a.tiles) {
      put_words<E>(a.link.states + rec * (64 * E) + lane, Ht);
      publish(a.link.flags + rec, 2u);
    }
  }
  __syncthreads();
  float h[E];
#pragma unroll
  for (int e = 0; e < E; ++e) h[e] = decay_step(decay_word(Gp[e]), sIn[e][lane], Hp[e]);
  static_assert(KDA_GATED_SCAN_CHUNK % S == 0, "a kept state stands in front of a wave's tokens");
  if (a.ckpt && t0 % KDA_GATED_SCAN_CHUNK == 0 && t0 < a.T && l.on) {
    const int chunks = (a.T + KDA_GATED_SCAN_CHUNK - 1) / KDA_GATED_SCAN_CHUNK;
#pragma unroll
    for (int e = 0; e < E; ++e) a.ckpt[((size_t)l.bh * chunks + t0 / KDA_GATED_SCAN_CHUNK) * a.D + l.d + e] = h[e];
  }
#pragma unroll
  for (int k = 0; k < S; ++k) {
#pragma unroll
    for (int e = 0; e < E; ++e) h[e] = decay_step(v[k][e], h[e], u[k][e]);
    if (full || t0 + k < l.n) scan_store<T, E>(a.y, base + k * row, h);
  }
  if (w == NW - 1 && tile.j + 1 == a.tiles && a.state_out && l.on)
#pragma unroll
    for (int e = 0; e < E; ++e) a.state_out[l.ch + e] = h[e];
}

template <typename T, int E, typename Off> void launch_e(const ScanArgs& a, hipStream_t s) {
  const unsigned grid = (unsigned)a.ctiles * (unsigned)a.tiles;
#define KDA_SCAN(G_, N_) scan_fwd_kernel<T, E, G_, N_, Off><<<grid, NW * 64, 0, s>>>(a)
  if (a.i) a.normalize ? KDA_SCAN(true, true) : KDA_SCAN(true, false);
  else a.normalize ? KDA_SCAN(false, true) : KDA_SCAN(false, false);
#undef KDA_SCAN
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
