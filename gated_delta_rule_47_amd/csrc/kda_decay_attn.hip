// Decay attention: the plan of segments, the join of the segments' states, the single-token step and
// the sequences of launches behind kda_decay_attn_fwd / _bwd (the walk itself: kda_decay_attn.h).
#include "kda_decay_attn.h"
#include "kda_launch.h"

namespace kda {

#define KDA_DECAY_EXTERN(T, KD)                \
  KDA_DECAY_FWD_INSTANCES(extern, T, KD)       \
  KDA_DECAY_BWD_INSTANCES(extern, T, KD)
KDA_DECAY_EXTERN(float, 32)
KDA_DECAY_EXTERN(float, 64)
KDA_DECAY_EXTERN(float, 128)
KDA_DECAY_EXTERN(bf16_t, 32)
KDA_DECAY_EXTERN(bf16_t, 64)
KDA_DECAY_EXTERN(bf16_t, 128)
#undef KDA_DECAY_EXTERN

// ------------------------------------------------------------------ segments
// A walk is sequential over its chunks, so heads x value tiles alone may leave most of the 256 CUs
// idle; then the tokens are cut into segments.  The price is a second read of k and v (the segments' local
// states) and two more launches.  The number of segments comes from a model in times of one chunk: workgroups
// run in rounds of one per CU; a round costs its chunks and a fixed part, a chunk of the pass over the state
// alone a share of a full one, the join and the launches a constant.  Measured, bf16, model in brackets:
// 1 x 4 heads of 30011 tokens, K = V = 128, forward: 24, 32, 40 segments 62, 56, 73 us (56, 48, 72); 2 x 16 heads of
// 8192: 1, 2, 3, 4 segments 120, 130, 107, 96 us (133, 126, 93, 75); backward, 8 x 8 heads of 4096, K = V = 64:
// 1, 2, 4 segments 65, 93, 91 us (69, 112, 106).  Four chunks at least in a segment, none in sequences of under 16.
// Of two plans within 5 % the one with more segments (a batch of unequal lengths spreads better).  fp32, 1 x 16 heads
// of 8191, K = V = 128: forward 1, 4, 8, 16 segments 573, 245, 165, 169 us, backward 1, 5, 8, 10 segments 576, 441, 424,
// 468.  The model counts one workgroup per CU also where a CU holds two (bf16, widths up to 64): 8 x 8 heads of 4096,
// K = V = 64, forward, 1, 2, 4, 8, 16 segments: 50, 59, 44, 44, 52 us, with lengths spread from 0 to 4096 49, 60, 41,
// 38, 43; it takes 4.
//
// A backward pass whose walks of dq and dk fill the chip once, and which with dv's would need half of a second
// round, gives dv's walk a launch of its own in two segments: dk's walk passes the state that the second
// one starts from, so that costs no pass over the state.  2 x 32 heads of 8192, K = V = 128, bf16: 381 us, all
// three in one launch 405, in two segments 457; from 8 bits 399, 453, 475; fp32, 1 x 43 heads of 4096: 635, 825, 734 (four
// segments 676).  Heads of up to 64 in both widths are left alone: bf16, of which a CU holds two, gains nothing by
// it (4 x 32 heads of 4096, K = V = 64: 135 and 137 us); fp32 would (483 and 417).  Where keys are narrow and values
// wide dv's two segments pass one round themselves, which the rule does not see: fp32, 65 heads of 4096, K = 8, V = 128
// take 449 us by it, in one launch 309.
DecayPlan decay_plan(int B, int H, int T, int K, int V, bool bf16, bool bwd) {
  const int C = bf16 ? 64 : 32;
  const int nchunks = (T + C - 1) / C;
  const long long fill = 256, wk = (long long)B * H * ((K + 63) / 64), wv = (long long)B * H * ((V + 63) / 64);
  const long long walks = bwd ? 2 * wk + wv : wv, states = bwd ? 2 * wv : wv;
  const double fixed = bf16 ? 5 : 3, join = bf16 ? 14 : 7, share = bf16 ? 0.6 : 0.35;
  const auto rounds = [&](long long blocks) { return (double)((blocks + fill - 1) / fill); };
  const auto cost = [&](long long n) {
    const double per = (double)((nchunks + n - 1) / n);
    const double walk = rounds(walks * n) * (per + fixed);
    return n == 1 ? walk : walk + rounds(states * (n - 1)) * (share * per + fixed) + join;
  };
  DecayPlan p{};
  int n = 1;
  if (nchunks >= 16) {
    double best = cost(1);
    for (int r = 1; r <= 3; ++r) {                           // as many as fill r rounds
      long long m = r * fill / walks;
      if (m > nchunks / 4) m = nchunks / 4;
      if (m > n && cost(m) < 1.05 * best) best = cost(m), n = (int)m;
    }
    if (bwd && (K > 64 || V > 64) && 2 * wk <= fill && walks > fill && 1.5 * nchunks + 3 * fixed < best)
      n = 1, p.vseg = 2;
  }
  const auto cut = [&](int n, int* seglen) {
    const int per = (nchunks + n - 1) / n;
    *seglen = (per < 1 ? 1 : per) * C;
    return nchunks ? (nchunks + per - 1) / per : 1;
  };
  p.nseg = cut(n, &p.seglen);
  p.vseg = cut(p.vseg ? p.vseg : 1, &p.vlen);
  return p;
}

size_t decay_states_bytes(int B, int H, int K, int V, const DecayPlan& p) {
  const int n = p.nseg > 1 ? p.nseg : p.vseg;
  return n > 1 ? (size_t)B * H * n * K * V * sizeof(float) : 0;
}

// Local end states -> states at the segments' starts, in place and in walking order:
// x[s] <- S, S <- a^{n_s} S + (old x[s]).  One thread per state element; the locals of 16 segments are
// fetched before the first is used, so the latency of memory is paid once in 16 (4 heads of 32 segments, K = V = 128:
// 8 us).  The first `nblock`
// workgroups join S, those behind them (a backward pass) dL/dS from the last segment on.
struct JoinArgs {
  float* x;
  const float* start;
};
__global__ void __launch_bounds__(256) decay_join_kernel(JoinArgs s, JoinArgs r, int nblock,
                                                         const float* __restrict__ log_decay,
                                                         const int* __restrict__ lengths, int H, int T, int nseg,
                                                         int seglen, int KV, int per_head) {
  constexpr int BATCH = 16;
  const bool rev = (int)blockIdx.x >= nblock;
  const int block = rev ? blockIdx.x - nblock : blockIdx.x;
  const JoinArgs a = rev ? r : s;
  const int bh = block / per_head, e = (block - bh * per_head) * 256 + threadIdx.x;
  if (e >= KV) return;
  int len = T;
  if (lengths) len = min(max(lengths[bh / H], 0), T);
  const float g = log_decay[bh % H];
  float* p = a.x + (size_t)bh * nseg * KV + e;
  float S = a.start ? a.start[(size_t)bh * KV + e] : 0.0f;
  DecaySteps whole(g, seglen);
  for (int s0 = 0; s0 < nseg; s0 += BATCH) {
    float loc[BATCH];
#pragma unroll
    for (int b = 0; b < BATCH; ++b) {
      const int i = s0 + b, seg = rev ? nseg - 1 - i : i;
      loc[b] = i < nseg - 1 ? p[(size_t)seg * KV] : 0.0f;    // the last one has no local state
    }
#pragma unroll
    for (int b = 0; b < BATCH; ++b) {
      const int i = s0 + b, seg = rev ? nseg - 1 - i : i;
      if (i < nseg) {
        p[(size_t)seg * KV] = S;
        const long long left = (long long)len - (long long)seg * seglen;
        const int n = left < 0 ? 0 : (left < seglen ? (int)left : seglen);
        S = fmaf(S, n == seglen ? whole.next() : decay_pow32(g, n), loc[b]);
      }
    }
  }
}

static hipError_t join(JoinArgs st, const JoinArgs* r, const float* log_decay, const int* lengths, int B, int H, int T,
                       int KV, const DecayPlan& p, hipStream_t s) {
  const int per_head = (KV + 255) / 256, n = B * H * per_head;
  hipLaunchKernelGGL(decay_join_kernel, dim3((unsigned)(r ? 2 * n : n)), dim3(256), 0, s, st, r ? *r : st, n, log_decay,
                     lengths, H, T, p.nseg, p.seglen, KV, per_head);
  return hipGetLastError();
}

template <typename T> static hipError_t walk_fwd(const WalkArgs& a, hipStream_t s) {
  if (a.K <= 32) return launch_walk_fwd<T, 32>(a, s);
  if (a.K <= 64) return launch_walk_fwd<T, 64>(a, s);
  return launch_walk_fwd<T, 128>(a, s);
}
template <typename T, int KD, bool PACK>
static hipError_t walk_bwd_v(const WalkArgs& dq, const WalkArgs& dk, const WalkArgs& dv, hipStream_t s) {
  if (dv.V <= 32) return launch_walk_bwd<T, KD, 32, PACK>(dq, dk, dv, s);
  if (dv.V <= 64) return launch_walk_bwd<T, KD, 64, PACK>(dq, dk, dv, s);
  return launch_walk_bwd<T, KD, 128, PACK>(dq, dk, dv, s);
}
template <typename T, bool PACK>
static hipError_t walk_bwd(const WalkArgs& dq, const WalkArgs& dk, const WalkArgs& dv, hipStream_t s) {
  if (dv.K <= 32) return walk_bwd_v<T, 32, PACK>(dq, dk, dv, s);
  if (dv.K <= 64) return walk_bwd_v<T, 64, PACK>(dq, dk, dv, s);
  return walk_bwd_v<T, 128, PACK>(dq, dk, dv, s);
}
template <typename T> static hipError_t segments(const SegArgs& st, const SegArgs* r, bool packed, hipStream_t s) {
  if (st.K <= 32) return launch_segments_kd<T, 32>(st, r, packed, s);
  if (st.K <= 64) return launch_segments_kd<T, 64>(st, r, packed, s);
  return launch_segments_kd<T, 128>(st, r, packed, s);
}

template <typename T>
hipError_t launch_decay_fwd(const void* q, const void* k, const void* v, const float* log_decay, const int* lengths,
                            const float* state_in, float scale, void* o, float* state_out, void* workspace, int B,
                            int H, int T_, int K, int V, hipStream_t s) {
  const DecayPlan p = decay_plan(B, H, T_, K, V, sizeof(T) == 2, false);
  float* ws = reinterpret_cast<float*>(workspace);
  if (p.nseg > 1) {
    const SegArgs g{k, v, nullptr, nullptr, log_decay, lengths, ws, 1.0f, B * H, H, T_, K, V, p.nseg, p.seglen,
                    state_out != nullptr};
    hipError_t e = segments<T>(g, nullptr, false, s);
    if (e == hipSuccess) e = join(JoinArgs{ws, state_in}, nullptr, log_decay, lengths, B, H, T_, K * V, p, s);
    if (e != hipSuccess) return e;
  }
  WalkArgs a{};
  a.q = q, a.k = k, a.v = v;
  a.log_decay = log_decay, a.lengths = lengths, a.state_in = state_in, a.seg_state = ws, a.state_out = state_out;
  a.returned = state_out != nullptr;
  a.o = o;
  a.c = a.r = scale, a.u = 1.0f;
  a.si_k = V, a.si_v = 1;
  a.BH = B * H, a.H = H, a.T = T_, a.K = K, a.V = V, a.nseg = p.nseg, a.seglen = p.seglen;
  return walk_fwd<T>(a, s);
}

// Segment boundaries and states are those of the K x V state in all three walks: S for dq, R = dL/dS
// for dk and dv, each computed and joined once.
template <typename T>
hipError_t launch_decay_bwd(const void* q, const void* k, const void* v, const uint8_t* q_sc, const uint8_t* k_sc,
                            const uint8_t* v_sc, const float* log_decay, const int* lengths, const float* state_in,
                            float scale, const void* d_o, const float* d_state_out, void* dq, void* dk, void* dv,
                            float* dstate_in, void* workspace, int B, int H, int T_, int K, int V, hipStream_t s) {
  const DecayPlan p = decay_plan(B, H, T_, K, V, sizeof(T) == 2, true);
  float* wS = reinterpret_cast<float*>(workspace);
  float* wR = wS + (p.nseg > 1 ? decay_states_bytes(B, H, K, V, p) / sizeof(float) : 0);
  const bool packed = q_sc != nullptr;                      // q, k and v, all or none
  hipError_t e = hipSuccess;
  if (p.nseg > 1) {
    const SegArgs gs{k, v, k_sc, v_sc, log_decay, lengths, wS, 1.0f, B * H, H, T_, K, V, p.nseg, p.seglen, false};
    const SegArgs gr{q, d_o, q_sc, nullptr, log_decay, lengths, wR, scale, B * H, H, T_, K, V, p.nseg, p.seglen, true};
    e = segments<T>(gs, &gr, packed, s);
    const JoinArgs jr{wR, d_state_out};
    if (e == hipSuccess) e = join(JoinArgs{wS, state_in}, &jr, log_decay, lengths, B, H, T_, K * V, p, s);
  }
  if (e != hipSuccess) return e;
  WalkArgs a{};
  a.log_decay = log_decay, a.lengths = lengths;
  a.BH = B * H, a.H = H, a.T = T_, a.nseg = p.nseg, a.seglen = p.seglen, a.zero_tail = lengths != nullptr;
  // dq: keys V, values K wide, the state read as its transpose
  WalkArgs dq_ = a;
  dq_.q = d_o, dq_.k = v, dq_.v = k, dq_.k_sc = v_sc, dq_.v_sc = k_sc;
  dq_.state_in = state_in, dq_.seg_state = wS, dq_.o = dq;
  dq_.c = dq_.r = scale, dq_.u = 1.0f;
  dq_.si_k = 1, dq_.si_v = V, dq_.K = V, dq_.V = K;
  WalkArgs dk_ = a;
  dk_.q = v, dk_.k = d_o, dk_.v = q, dk_.q_sc = v_sc, dk_.v_sc = q_sc;
  dk_.state_in = d_state_out, dk_.seg_state = wR, dk_.o = dk;
  dk_.c = dk_.u = scale, dk_.r = 1.0f;
  dk_.si_k = 1, dk_.si_v = V, dk_.K = V, dk_.V = K;
  // dv, and the state's gradient
  WalkArgs dv_ = a;
  dv_.q = k, dv_.k = q, dv_.v = d_o, dv_.q_sc = k_sc, dv_.k_sc = q_sc;
  dv_.state_in = d_state_out, dv_.seg_state = wR, dv_.state_out = dstate_in, dv_.o = dv;
  dv_.c = dv_.u = scale, dv_.r = 1.0f;
  dv_.si_k = V, dv_.si_v = 1, dv_.K = K, dv_.V = V;
  dv_.returned = dstate_in != nullptr;
  if (p.vseg > 1) {
    dk_.mid = wR, dk_.nmid = dv_.nseg = p.vseg, dk_.midlen = dv_.seglen = p.vlen;
    dk_.returned = dv_.returned;
  }
  return packed ? walk_bwd<T, true>(dq_, dk_, dv_, s) : walk_bwd<T, false>(dq_, dk_, dv_, s);
}

// ------------------------------------------------------------------ one token
// S <- a S + k v^T and o = scale S^T q for one token per head.  Bound by the state's traffic (2 K V
// fp32 per head): a thread holds four columns (one 16-byte access) of K / RG rows, all loaded before
// the first is used; the RG partial sums of a column meet in LDS.  VS columns per workgroup.  The decay is taken
// as hi + lo: rounded to fp32 it would be off to the same side in every call of a long answer (1e-4 of the state
// after 4096 of them).
// bf16, K = V = 128: 192 x 32 heads 157 to 162 us (5.0 to 5.2 TB/s; fp32 161), 4 x 32 heads 4.6 us, where a launch alone
// takes as long.
template <typename T, int VS>
__global__ void __launch_bounds__(256) decay_step_kernel(const T* __restrict__ q, const T* __restrict__ k,
                                                         const T* __restrict__ v,
                                                         const float* __restrict__ log_decay,
                                                         float* __restrict__ state, float scale, T* __restrict__ o,
                                                         int H, int K, int V) {
  constexpr int LC = VS / 4, RG = 256 / LC, MAXR = (128 + RG - 1) / RG;
  __shared__ float sq[128], sk[128];
  __shared__ __align__(16) float red[RG * VS];
  const int ntile = V / VS;
  const int bh = blockIdx.x / ntile, v0 = (blockIdx.x - bh * ntile) * VS;
  const int tid = threadIdx.x, c = tid % LC, rg = tid / LC;
  float* S = state + (size_t)bh * K * V + v0 + 4 * c;
  floatx4 s[MAXR];
#pragma unroll
  for (int i = 0; i < MAXR; ++i) {
    const int row = rg + i * RG;
    if (row < K) s[i] = *reinterpret_cast<const floatx4*>(S + (size_t)row * V);
  }
  if (tid < K) {
    sq[tid] = to_f<T>(q[(size_t)bh * K + tid]);
    sk[tid] = to_f<T>(k[(size_t)bh * K + tid]);
  }
  const DecaySteps a(log_decay[bh % H], 1);
  const T* vp = v + (size_t)bh * V + v0 + 4 * c;
  const floatx4 vv = {to_f<T>(vp[0]), to_f<T>(vp[1]), to_f<T>(vp[2]), to_f<T>(vp[3])};
  lds_barrier();
  floatx4 sum = zero4();
#pragma unroll
  for (int i = 0; i < MAXR; ++i) {
    const int row = rg + i * RG;
    if (row < K) {
      const float kr = sk[row], qr = sq[row];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        // (an infinite state times lo = 0, or of lo's sign, would be NaN)
        const float fin = __builtin_amdgcn_fmed3f(s[i][e], -3.0e38f, 3.0e38f);
        s[i][e] = fmaf(a.hi, s[i][e], fmaf(a.lo, fin, kr * vv[e]));
        sum[e] = fmaf(qr, s[i][e], sum[e]);
      }
      *reinterpret_cast<floatx4*>(S + (size_t)row * V) = s[i];
    }
  }
  *reinterpret_cast<floatx4*>(red + rg * VS + 4 * c) = sum;
  lds_barrier();
  if (tid < VS) {
    float x = 0.0f;
#pragma unroll
    for (int r = 0; r < RG; ++r) x += red[r * VS + tid];
    o[(size_t)bh * V + v0 + tid] = from_f<T>(scale * x);
  }
}

template <typename T>
hipError_t launch_decay_step(const void* q, const void* k, const void* v, const float* log_decay, float* state,
                             float scale, void* o, int B, int H, int K, int V, hipStream_t s) {
#define KDA_DECAY_STEP(VS)                                                                                          \
  hipLaunchKernelGGL((decay_step_kernel<T, VS>), dim3((unsigned)(B * H * (V / VS))), dim3(256), 0, s, (const T*)q,  \
                     (const T*)k, (const T*)v, log_decay, state, scale, (T*)o, H, K, V)
  if (V >= 32) KDA_DECAY_STEP(32);
  else if (V == 16) KDA_DECAY_STEP(16);
  else KDA_DECAY_STEP(8);
#undef KDA_DECAY_STEP
  return hipGetLastError();
}

#define KDA_INST(T)                                                                                                  \
  template hipError_t launch_decay_fwd<T>(const void*, const void*, const void*, const float*, const int*,           \
                                          const float*, float, void*, float*, void*, int, int, int, int, int,        \
                                          hipStream_t);                                                              \
  template hipError_t launch_decay_bwd<T>(const void*, const void*, const void*, const uint8_t*, const uint8_t*,     \
                                          const uint8_t*, const float*, const int*, const float*, float,             \
                                          const void*, const float*, void*, void*, void*, float*, void*, int, int,   \
                                          int, int, int, hipStream_t);                                               \
  template hipError_t launch_decay_step<T>(const void*, const void*, const void*, const float*, float*, float,       \
                                           void*, int, int, int, int, hipStream_t);
KDA_INST(float)
KDA_INST(bf16_t)
#undef KDA_INST

}  // namespace kda
