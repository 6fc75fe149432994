// Norm of every head's query and key with the rotation by the token's position in the same pass, and its adjoint.
//
//   r = (mean x^2 + eps)^-1/2 or (sum x^2 + eps)^-1/2 or 1,  y = Rot(x r w)
//   p = Rot^T dy,  xh = x r,  dx = r (p w - xh mean(p w xh)) (the sum for the l2 norm),  dw = sum over rows of p xh
//   Rot turns the pair (u, v) of every rotated pair of channels by position * frequency, times a scale.
//
// Memory bounds it: every row is read once and written once.  Rows are read token by token, as a fused projection
// leaves them (any strides), and written head by head, as attention reads them.  A lane holds eight channels of a row in
// two groups of four, chosen so that both channels of a pair are its own: 4 i and R / 2 + 4 i for pairs half a rotated
// part apart, 8 i and 8 i + 4 otherwise.  It stays on its channels and goes over the heads of its token, so an angle is
// computed once per token and chunk of heads.
//
// An angle is position * frequency in float64, reduced to a part of a turn there (a position of 2^20 at a frequency
// of 1 has 17 bits in front of the point and needs 24 behind it), then sine and cosine in float32.
// Measured: forward, 16384 tokens of 2 x 32 heads of 128, bf16, 112 us (4.8 TB/s), heads of 64 the same rate, of 80 (ten of sixteen
// lanes) 4.2 TB/s; adjoint, 2 x 8192 such tokens, 168 us and 5 for the sums (4.65 TB/s); 192 tokens of 40 heads 4.8 us.
#include "kda_launch.h"
#include "kda_vec.h"

namespace kda {
namespace {

constexpr int kQkThreads = 256;

struct QkSide {                     // queries or keys
  const void* x;
  long long xb, xt, xh;             // strides in elements
  const float* w;                   // (Hw, D), Hw = 1 or H
  void* y;                          // forward: (B, H, T, D) out; backward: the cotangent
  void* dx;
  long long db, dt, dh;
  float* parts;                     // backward: (heads' chunks, token blocks, D)
  int H, chunk, per_head;           // heads of a workgroup; w has a row per head
};
struct QkArgs {
  QkSide side[2];
  const double* freqs;              // (R / 2)
  const int* positions;             // (B, T)
  float eps, inv_n, rope_scale;
  int B, T, D, R, norm, q_chunks, tokens, blocks;   // token blocks per workgroup, workgroups along the tokens
};

// The two groups of four channels of item i, and whether they are rotated.
struct QkItem {
  int o0, o1;
  bool on, rot;
};
template <bool INTER> __device__ __forceinline__ QkItem qk_item(int i, int D, int R) {
  QkItem q;
  q.on = 8 * i < D;
  q.rot = 8 * i < R;
  const bool half = !INTER && q.rot;
  q.o0 = half ? 4 * i : 8 * i;
  q.o1 = half ? R / 2 + 4 * i : 8 * i + 4;
  return q;
}

// cos and sin of the four pairs of item i at a position.
__device__ __forceinline__ void qk_angles(const double* freqs, int i, int pos, float scale, float (&c)[4], float (&s)[4]) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const double turns = (double)pos * freqs[4 * i + e] * 0.15915494309189533577;   // 1 / (2 pi)
    const float part = (float)(turns - __builtin_rint(turns));
    sincospif(2.0f * part, &s[e], &c[e]);
    s[e] *= scale;
    c[e] *= scale;
  }
}

// f: the item's eight channels; SIGN = -1 turns back.
template <bool INTER, int SIGN> __device__ __forceinline__ void qk_turn(float (&f)[8], const float (&c)[4], const float (&s)[4]) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    float& u = f[INTER ? 2 * e : e];
    float& v = f[INTER ? 2 * e + 1 : 4 + e];
    const float a = u, b = v, t = SIGN * s[e];
    u = a * c[e] - b * t;
    v = b * c[e] + a * t;
  }
}

template <typename T> struct QkRow {
  Elems<T, 4> a, b;
  __device__ __forceinline__ void load(const T* p, const QkItem& q) {
    a.load(p + q.o0);
    b.load(p + q.o1);
  }
  __device__ __forceinline__ void zero() {
    a.zero();
    b.zero();
  }
  __device__ __forceinline__ void get(float (&f)[8]) const {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      f[e] = a.at(e);
      f[4 + e] = b.at(e);
    }
  }
  __device__ __forceinline__ void put(T* p, const QkItem& q, const float (&f)[8]) {
    a.set(f);
    b.set(f + 4);
    a.store(p + q.o0);
    b.store(p + q.o1);
  }
};

__device__ __forceinline__ void qk_weight(const float* w, const QkItem& q, float (&f)[8]) {
  if (w && q.on) {
    load_f32<4>(w + q.o0, f);
    load_f32<4>(w + q.o1, f + 4);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = 1.f;
  }
}

// The side and the heads of a workgroup: chunk c of the queries' and then the keys' chunks.
struct QkHeads {
  int side, h0, h1, chunk;
};
__device__ __forceinline__ QkHeads qk_heads(const QkArgs& a, unsigned c) {
  QkHeads h;
  h.side = c >= (unsigned)a.q_chunks;
  h.chunk = (int)c - (h.side ? a.q_chunks : 0);
  const QkSide& s = a.side[h.side];
  h.h0 = h.chunk * s.chunk;
  h.h1 = min(h.h0 + s.chunk, s.H);
  return h;
}

// L lanes per row (a power of two, 8 L >= D); U rows of a lane in flight.
template <typename T, int L, bool INTER> __global__ __launch_bounds__(kQkThreads) void qk_fwd_kernel(QkArgs a) {
  constexpr int U = 4, TB = kQkThreads / L;
  const int i = threadIdx.x & (L - 1);
  const QkItem it = qk_item<INTER>(i, a.D, a.R);
  const unsigned tb = blockIdx.x % (unsigned)a.blocks;
  const QkHeads hs = qk_heads(a, blockIdx.x / (unsigned)a.blocks);
  const QkSide& sd = a.side[hs.side];
  const size_t yh = (size_t)a.T * a.D;
  float w[8];
  qk_weight(sd.w, it, w);
  for (int k = 0; k < a.tokens; ++k) {
    const long long at = ((long long)tb * a.tokens + k) * TB + threadIdx.x / L;
    const bool on = at < a.B * a.T && it.on;
    const int tok = on ? (int)at : 0, b = tok / a.T, t = tok - b * a.T;
    float c[4], s[4];
    if (on && it.rot) qk_angles(a.freqs, i, a.positions ? a.positions[tok] : t, a.rope_scale, c, s);
    const T* x = (const T*)sd.x + b * sd.xb + t * sd.xt + hs.h0 * sd.xh;
    T* y = (T*)sd.y + (((size_t)b * sd.H + hs.h0) * a.T + t) * a.D;
    for (int h = hs.h0; h < hs.h1; h += U, x += U * sd.xh, y += U * yh) {
      QkRow<T> raw[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        raw[u].zero();
        if (on && h + u < hs.h1) raw[u].load(x + u * sd.xh, it);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (h + u >= hs.h1) break;
        float f[8];
        raw[u].get(f);
        if (a.norm) {
          float sq = 0.f;
#pragma unroll
          for (int e = 0; e < 8; ++e) sq = fmaf(f[e], f[e], sq);
          const float r = rsqrtf(fmaf(lane_sum<L>(sq), a.inv_n, a.eps));
          if (sd.per_head) qk_weight(sd.w + (size_t)(h + u) * a.D, it, w);
#pragma unroll
          for (int e = 0; e < 8; ++e) f[e] *= r * w[e];
        }
        if (it.rot) qk_turn<INTER, 1>(f, c, s);
        if (on) raw[u].put(y + u * yh, it, f);
      }
    }
  }
}

// A workgroup takes a.tokens blocks of TB tokens of its heads; the weights' gradient is summed in registers over
// them (one head only where every head has weights of its own), then over the lanes of a channel.
template <typename T, int L, bool INTER> __global__ __launch_bounds__(kQkThreads) void qk_bwd_kernel(QkArgs a) {
  constexpr int U = 2, TB = kQkThreads / L;
  __shared__ float red[kQkThreads * 8];
  const int i = threadIdx.x & (L - 1);
  const QkItem it = qk_item<INTER>(i, a.D, a.R);
  const unsigned tb = blockIdx.x % (unsigned)a.blocks;
  const QkHeads hs = qk_heads(a, blockIdx.x / (unsigned)a.blocks);
  const QkSide& sd = a.side[hs.side];
  const size_t yh = (size_t)a.T * a.D;
  float w[8], dw[8];
  qk_weight(sd.w && sd.per_head ? sd.w + (size_t)hs.h0 * a.D : sd.w, it, w);      // (a row per head without weights: ones)
#pragma unroll
  for (int e = 0; e < 8; ++e) dw[e] = 0.f;
  for (int k = 0; k < a.tokens; ++k) {
    const long long at = ((long long)tb * a.tokens + k) * TB + threadIdx.x / L;
    const bool on = at < a.B * a.T && it.on;
    const int tok = on ? (int)at : 0, b = tok / a.T, t = tok - b * a.T;
    float c[4], s[4];
    if (on && it.rot) qk_angles(a.freqs, i, a.positions ? a.positions[tok] : t, a.rope_scale, c, s);
    const T* x = (const T*)sd.x + b * sd.xb + t * sd.xt + hs.h0 * sd.xh;
    const T* dy = (const T*)sd.y + (((size_t)b * sd.H + hs.h0) * a.T + t) * a.D;
    T* dx = (T*)sd.dx + b * sd.db + t * sd.dt + hs.h0 * sd.dh;
    for (int h = hs.h0; h < hs.h1; h += U, x += U * sd.xh, dy += U * yh, dx += U * sd.dh) {
      QkRow<T> rx[U], rd[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        rx[u].zero();
        rd[u].zero();
        if (on && h + u < hs.h1) {
          rd[u].load(dy + u * yh, it);
          if (a.norm) rx[u].load(x + u * sd.xh, it);
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (h + u >= hs.h1) break;
        float p[8];
        rd[u].get(p);
        if (it.rot) qk_turn<INTER, -1>(p, c, s);
        if (a.norm) {
          float f[8], sq = 0.f, dot = 0.f;
          rx[u].get(f);
#pragma unroll
          for (int e = 0; e < 8; ++e) sq = fmaf(f[e], f[e], sq);
          const float r = rsqrtf(fmaf(lane_sum<L>(sq), a.inv_n, a.eps));
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            f[e] *= r;
            if (on) dw[e] = fmaf(p[e], f[e], dw[e]);
            p[e] *= w[e];
            dot = fmaf(p[e], f[e], dot);
          }
          dot = lane_sum<L>(dot) * a.inv_n;
#pragma unroll
          for (int e = 0; e < 8; ++e) p[e] = r * fmaf(-f[e], dot, p[e]);
        }
        if (on) rx[u].put(dx + u * sd.dh, it, p);
      }
    }
  }
  if (!sd.parts) return;
#pragma unroll
  for (int e = 0; e < 8; ++e) red[e * kQkThreads + threadIdx.x] = dw[e];
  __syncthreads();
  float* out = sd.parts + ((size_t)hs.chunk * a.blocks + tb) * a.D;
  for (int k = threadIdx.x; k < L * 8; k += kQkThreads) {
    const int j = k & (L - 1), e = k / L;
    const QkItem jt = qk_item<INTER>(j, a.D, a.R);
    float sum = 0.f;
    for (int r = 0; r < TB; ++r) sum += red[e * kQkThreads + r * L + j];
    if (jt.on) out[(e < 4 ? jt.o0 : jt.o1 - 4) + e] = sum;
  }
}

// Row blockIdx.y of the weights' gradients, the queries' rows and then the keys': the sum of its workgroups' parts.
struct QkSums {
  const float* in[2];
  float* out[2];
  int rows[2], parts[2];            // rows: 1, or the heads
};
__global__ __launch_bounds__(kSumThreads) void qk_params_kernel(QkSums q, int D) {
  const int side = (int)blockIdx.y >= q.rows[0];
  const size_t h = blockIdx.y - (side ? q.rows[0] : 0);
  float* out = q.out[side] + h * D;
  sum_parts(q.in[side] + h * q.parts[side] * D, D, q.parts[side], D, [=](int i, float s) { out[i] = s; });
}

int lanes_of(int D) {
  int L = 1;
  while (8 * L < D) L *= 2;
  return L;
}

// Heads per workgroup: the angles of a token and item cost about as much as two rows of it, so up to eight heads
// share them where that still leaves 2048 workgroups (eight per CU).
int head_chunk(long long token_blocks, int heads) {
  int c = 8;
  while (c > 1 && token_blocks * ((heads + c - 1) / c) < 2048) c /= 2;
  return c;
}
int chunks(const QkSide& s) { return s.H ? (s.H + s.chunk - 1) / s.chunk : 0; }

// Chunks of heads and blocks of tokens; backward, blocks per workgroup: as many as leave 1024 workgroups, up to 32,
// since each workgroup adds a part to the weights' gradient (2048: 178 us for 173 at 2 x 8192 tokens of 2 x 32 heads of 128) (and so many that the grid keeps within 2^22).
void qk_plan(QkArgs& a, bool bwd) {
  const int TB = kQkThreads / lanes_of(a.D);
  const long long n = ((long long)a.B * a.T + TB - 1) / TB;
  for (QkSide& s : a.side) s.chunk = s.per_head && bwd ? 1 : head_chunk(n, a.side[0].H + a.side[1].H);
  a.q_chunks = chunks(a.side[0]);
  const long long c = a.q_chunks + chunks(a.side[1]);
  a.tokens = 1;
  while ((bwd && a.tokens < 32 && n / (2 * a.tokens) * c >= 1024) || n / a.tokens * c > (1 << 22)) a.tokens *= 2;
  a.blocks = (int)((n + a.tokens - 1) / a.tokens);
}

template <typename T, bool INTER> hipError_t launch_qk(const QkArgs& a, bool bwd, hipStream_t s) {
  const unsigned grid = (unsigned)((long long)a.blocks * (a.q_chunks + chunks(a.side[1])));
#define KDA_QK(L)                                                           \
  case L:                                                                   \
    if (bwd) qk_bwd_kernel<T, L, INTER><<<grid, kQkThreads, 0, s>>>(a);     \
    else qk_fwd_kernel<T, L, INTER><<<grid, kQkThreads, 0, s>>>(a);         \
    break;
  switch (lanes_of(a.D)) {
    KDA_QK(1) KDA_QK(2) KDA_QK(4) KDA_QK(8) KDA_QK(16) KDA_QK(32)
    default: return hipErrorInvalidValue;
  }
#undef KDA_QK
  return hipGetLastError();
}

QkArgs qk_args(const QkSideDesc* d, const double* freqs, const int* positions, int norm, float eps, float rope_scale,
               int B, int T, int D, int R, bool bwd) {
  QkArgs a = {};
  for (int i = 0; i < 2; ++i) {
    QkSide& s = a.side[i];
    s.x = d[i].x, s.xb = d[i].xb, s.xt = d[i].xt, s.xh = d[i].xh, s.w = d[i].w, s.y = d[i].y, s.H = d[i].H;
    s.dx = d[i].dx, s.db = d[i].db, s.dt = d[i].dt, s.dh = d[i].dh;
    s.per_head = d[i].per_head;
  }
  a.freqs = freqs, a.positions = positions, a.norm = norm, a.eps = eps, a.rope_scale = rope_scale;
  a.inv_n = norm == 1 ? 1.0f / D : 1.0f;
  a.B = B, a.T = T, a.D = D, a.R = R;
  qk_plan(a, bwd);
  return a;
}

}  // namespace

template <typename T>
hipError_t launch_qk_fwd(const QkSideDesc* d, const double* freqs, const int* positions, int norm, float eps,
                         float rope_scale, int interleaved, int B, int T_, int D, int R, hipStream_t s) {
  if (T_ == 0) return hipSuccess;
  const QkArgs a = qk_args(d, freqs, positions, norm, eps, rope_scale, B, T_, D, R, false);
  return interleaved ? launch_qk<T, true>(a, false, s) : launch_qk<T, false>(a, false, s);
}

size_t qk_bwd_workspace_bytes(int B, int T, int Hq, int Hk, int D, int q_per_head, int k_per_head) {
  QkSideDesc d[2] = {};
  d[0].H = Hq, d[1].H = Hk, d[0].per_head = q_per_head, d[1].per_head = k_per_head;
  const QkArgs a = qk_args(d, nullptr, nullptr, 0, 0.f, 1.f, B, T, D, 0, true);
  return (size_t)(a.q_chunks + chunks(a.side[1])) * a.blocks * D * 4;
}

template <typename T>
hipError_t launch_qk_bwd(const QkSideDesc* d, const double* freqs, const int* positions, int norm, float eps,
                         float rope_scale, int interleaved, float* dwq, float* dwk, void* workspace, int B, int T_,
                         int D, int R, hipStream_t s) {
  QkArgs a = qk_args(d, freqs, positions, norm, eps, rope_scale, B, T_, D, R, true);
  if (dwq) a.side[0].parts = (float*)workspace;
  if (dwk) a.side[1].parts = (float*)workspace + (size_t)a.q_chunks * a.blocks * D;
  if (T_) {
    const hipError_t e = interleaved ? launch_qk<T, true>(a, true, s) : launch_qk<T, false>(a, true, s);
    if (e != hipSuccess) return e;
  }
  float* dw[2] = {dwq, dwk};
  QkSums q = {};
  for (int i = 0; i < 2; ++i) {
    if (!dw[i]) continue;
    const QkSide& sd = a.side[i];
    q.in[i] = sd.parts, q.out[i] = dw[i];
    q.rows[i] = sd.per_head ? sd.H : 1, q.parts[i] = (sd.per_head ? 1 : chunks(sd)) * a.blocks;
  }
  if (q.rows[0] + q.rows[1] == 0) return hipSuccess;
  qk_params_kernel<<<dim3((D + 63) / 64, q.rows[0] + q.rows[1]), kSumThreads, 0, s>>>(q, D);
  return hipGetLastError();
}

#define KDA_QK_INST(T)                                                                                                \
  template hipError_t launch_qk_fwd<T>(const QkSideDesc*, const double*, const int*, int, float, float, int, int, int, \
                                       int, int, hipStream_t);                                                        \
  template hipError_t launch_qk_bwd<T>(const QkSideDesc*, const double*, const int*, int, float, float, int, float*,  \
                                       float*, void*, int, int, int, int, hipStream_t);
KDA_QK_INST(float)
KDA_QK_INST(bf16_t)

}  // namespace kda
