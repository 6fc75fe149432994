// Adjoint of the gated recurrence (kda_gated_scan.h has the mathematics and the way tiles are linked).  Tiles run from
// the last token to the first; r crosses them as the state does forward.  h comes from the kept state in front of the
// tile, one row per tile, so a tile needs its predecessors in one direction only.
#include "kda_gated_scan.h"

#include "../../include/kda.h"

namespace kda {
namespace {

constexpr int NW = kScanBwdWaves, S = kScanBwdTokens;
static_assert(NW * S == KDA_GATED_SCAN_CHUNK, "one kept state per tile");

template <typename T, int E, bool GATE, bool NORM, typename Off>
__global__ __launch_bounds__(NW * 64) __attribute__((amdgpu_waves_per_eu(3))) void scan_bwd_kernel(ScanArgs a) {
  __shared__ uint32_t slot;
  __shared__ float sG[NW][E][64], sH[NW][E][64], sR[NW][E][64], sIn[E][64];
  const ScanTile tile = scan_tile(a, &slot);
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const ScanLane<E> l = scan_lane<E>(a, tile.c, lane);
  const int jt = a.tiles - 1 - tile.j;     // place in time
  const int t0 = (jt * NW + w) * S;
  const Off row = (Off)a.D * sizeof(T);
  const Off base = ((Off)l.bh * a.T + t0) * a.D * sizeof(T) + (Off)l.d * sizeof(T);
  const bool full = __all(t0 + S <= l.n);

  ScanRaw<T, E> rz[S], rx[S], ri[S], rd[S];
  if (full) {
#pragma unroll
    for (int k = 0; k < S; ++k) {
      rz[k].load(a.z, base + k * row);
      rx[k].load(a.x, base + k * row);
      if constexpr (GATE) ri[k].load(a.i, base + k * row);
      rd[k].load(a.dy, base + k * row);
    }
  } else {
#pragma unroll
    for (int k = 0; k < S; ++k) {
      rz[k].u = rx[k].u = ri[k].u = rd[k].u = 0;
      if (t0 + k < l.n) {
        rz[k].load(a.z, base + k * row);
        rx[k].load(a.x, base + k * row);
        if constexpr (GATE) ri[k].load(a.i, base + k * row);
        rd[k].load(a.dy, base + k * row);
      }
    }
  }
  float h0[E];
#pragma unroll
  for (int e = 0; e < E; ++e) h0[e] = l.on && jt * NW * S < a.T ? a.ckpt[((size_t)l.bh * a.tiles + jt) * a.D + l.d + e] : 0.f;

  // per token: the decay v, g2, q = m sigmoid(z'), c = n s, sm = 1 - s, k4 = a^2 s x / n
  float v[S][E], g[S][E], q[S][E], c[S][E], sm[S][E], k4[S][E], G[E], H[E], R[E];
#pragma unroll
  for (int e = 0; e < E; ++e) G[e] = H[e] = R[e] = 0.f;
#pragma unroll
  for (int k = 0; k < S; ++k)
#pragma unroll
    for (int e = 0; e < E; ++e) {
      float y;
      const float p = fmaf(rz[k].at(e), kLog2e, l.bias2[e]);
      g[k][e] = -l.m * scan_softplus2(p, y);
      q[k][e] = l.m * fast_rcp(1.f + y) * (p >= 0.f ? 1.f : y);
      v[k][e] = decay_word(g[k][e]);
      const float s = GATE ? scan_sigmoid(ri[k].at(e)) : 1.f, x = rx[k].at(e);
      sm[k][e] = 1.f - s;
      c[k][e] = s;
      k4[k][e] = 0.f;
      if constexpr (NORM) {
        // n = 0 (a decay of exactly 1): 1 / n is held at 1e18, and q = 0 or tiny takes the term to its limit 0 in dz
        const float n2 = decay_n2(v[k][e]), rn = __builtin_amdgcn_rsqf(fmaxf(n2, 1e-36f)), av = decay_a(v[k][e]);
        c[k][e] = s * (n2 * rn);
        k4[k][e] = av * av * rn * (s * x);
      }
      if (!full && t0 + k >= l.n) {        // behind the sequence: the state stays, nothing has a gradient
        v[k][e] = kNoDecay;
        g[k][e] = q[k][e] = c[k][e] = k4[k][e] = 0.f;
      }
      G[e] += g[k][e];
      H[e] = decay_step(v[k][e], H[e], c[k][e] * x);
    }
#pragma unroll
  for (int k = S - 1; k >= 0; --k)
#pragma unroll
    for (int e = 0; e < E; ++e) R[e] = decay_step(v[k][e], R[e] + rd[k].at(e), 0.f);
#pragma unroll
  for (int e = 0; e < E; ++e) {
    sG[w][e][lane] = G[e];
    sH[w][e][lane] = H[e];
    sR[w][e][lane] = R[e];
  }
  __syncthreads();
  // h in front of this wave's tokens; r behind them from a zero behind the tile
  float h[E], Gs[E], Rs[E];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    h[e] = h0[e];
    for (int p = 0; p < w; ++p) h[e] = decay_step(decay_word(sG[p][e][lane]), h[e], sH[p][e][lane]);
    Gs[e] = Rs[e] = 0.f;
    for (int p = NW - 1; p > w; --p) {
      Rs[e] = decay_step(decay_word(sG[p][e][lane]), Rs[e], sR[p][e][lane]);
      Gs[e] += sG[p][e][lane];
    }
  }
  if (w == 0) {
    float Gt[E], Rt[E], in[E];
    const size_t first = (size_t)tile.c * a.tiles, rec = first + tile.j;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      Rt[e] = decay_step(decay_word(G[e]), Rs[e], R[e]);
      Gt[e] = Gs[e] + G[e];
      in[e] = 0.f;
    }
    if (tile.j == 0) {
      if (a.d_state && l.on)
#pragma unroll
        for (int e = 0; e < E; ++e) in[e] = a.d_state[l.ch + e];
    } else {
      float* pair = a.link.pairs + rec * (128 * E) + lane;
      put_words<E>(pair, Gt);
      put_words<E>(pair + 64 * E, Rt);
      publish(a.link.flags + rec, 1u);
      look_back<E>(a.link, first, tile.j, lane, in);
    }
#pragma unroll
    for (int e = 0; e < E; ++e) {
      sIn[e][lane] = in[e];
      Rt[e] = decay_step(decay_word(Gt[e]), in[e], Rt[e]);
    }
    if (tile.j + 1 < a.tiles) {
      put_words<E>(a.link.states + rec * (64 * E) + lane, Rt);
      publish(a.link.flags + rec, 2u);
    } else if (l.on) {
#pragma unroll
      for (int e = 0; e < E; ++e) a.d_state_in[l.ch + e] = Rt[e];
    }
  }
  // dg / r = a h_{t-1} - a^2 s x / n of every token
#pragma unroll
  for (int k = 0; k < S; ++k)
#pragma unroll
    for (int e = 0; e < E; ++e) {
      k4[k][e] = fmaf(decay_a(v[k][e]), h[e], -k4[k][e]);
      h[e] = decay_step(v[k][e], h[e], c[k][e] * rx[k].at(e));
    }
  __syncthreads();
  float r[E], sz[E], sa[E];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    r[e] = decay_step(decay_word(Gs[e]), sIn[e][lane], Rs[e]);
    sz[e] = sa[e] = 0.f;
  }
#pragma unroll
  for (int k = S - 1; k >= 0; --k) {
    float dx[E], dz[E], di[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
      r[e] += rd[k].at(e);
      dx[e] = r[e] * c[k][e];
      di[e] = dx[e] * rx[k].at(e) * sm[k][e];
      const float dg = r[e] * k4[k][e];
      dz[e] = -dg * q[k][e];
      if (!full && t0 + k >= l.n) dx[e] = di[e] = dz[e] = 0.f;
      else {
        sz[e] += dz[e];
        sa[e] = fmaf(dg, g[k][e], sa[e]);
      }
      r[e] = decay_step(v[k][e], r[e], 0.f);
    }
    if (full || (l.on && t0 + k < a.T)) {
      scan_store<T, E>(a.dx, base + k * row, dx);
      scan_store<T, E>(a.dz, base + k * row, dz);
      if constexpr (GATE) scan_store<T, E>(a.di, base + k * row, di);
    }
  }
  if (!a.parts) return;
  // the waves' sums in a fixed order (the exchange's arrays are free: every wave has read them before the barrier)
#pragma unroll
  for (int e = 0; e < E; ++e) {
    sG[w][e][lane] = sz[e];
    sH[w][e][lane] = sa[e] * kLn2;
  }
  __syncthreads();
  if (w == 0 && l.on) {
    const size_t N = (size_t)a.B * a.H * a.D;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      float z = 0.f, s = 0.f;
#pragma unroll
      for (int p = 0; p < NW; ++p) {
        z += sG[p][e][lane];
        s += sH[p][e][lane];
      }
      a.parts[(size_t)jt * N + l.ch + e] = z;
      a.parts[((size_t)a.tiles + jt) * N + l.ch + e] = s;
    }
  }
}

template <typename T, int E, typename Off> void launch_e(const ScanArgs& a, hipStream_t s) {
  const unsigned grid = (unsigned)a.ctiles * (unsigned)a.tiles;
#define KDA_SCAN(G_, N_) scan_bwd_kernel<T, E, G_, N_, Off><<<grid, NW * 64, 0, s>>>(a)
  if (a.i) a.normalize ? KDA_SCAN(true, true) : KDA_SCAN(true, false);
  else a.normalize ? KDA_SCAN(false, true) : KDA_SCAN(false, false);
#undef KDA_SCAN
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
