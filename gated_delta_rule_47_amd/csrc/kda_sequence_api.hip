// C ABI of the short convolution, the query and key norm with rotation and the gated recurrence (see
// include/kda.h): argument checks, status codes, dispatch by type.  Nothing is launched before every check has passed.
#include <math.h>
#include <stdint.h>

#include "../../include/kda.h"
#include "kda_launch.h"

namespace kda {
namespace {

typedef long long ll;
constexpr ll kMostElements = 1LL << 48;

bool valid_dtype(int t) { return t == KDA_F32 || t == KDA_BF16; }
size_t esize(int dtype) { return dtype == KDA_BF16 ? 2 : 4; }
bool aligned(const void* p, size_t n) { return ((uintptr_t)p & (n - 1)) == 0; }

// A buffer of rows: `row` bytes at every place i0 * s[0] + i1 * s[1] + i2 * s[2] (bytes; batch, token, head), ik < n[k].
struct Rows {
  const void* p;
  ll row, n[3], s[3];
  bool none() const { return !p || row <= 0 || n[0] <= 0 || n[1] <= 0 || n[2] <= 0; }
  ll span() const { return (n[0] - 1) * s[0] + (n[1] - 1) * s[1] + (n[2] - 1) * s[2] + row; }
};
Rows flat(const void* p, ll bytes) { return {p, bytes, {1, 1, 1}, {0, 0, 0}}; }

// Whether b, which starts `off` bytes behind a, lies beside it within a period that both share: one dimension k whose
// stride holds what either covers in its smaller dimensions side by side, and larger dimensions that both share too and
// whose strides hold all the periods inside them.
bool beside(const Rows& a, const Rows& b, ll off) {
  for (int k = 0; k < 3; ++k) {
    if (a.n[k] < 2 || a.n[k] != b.n[k] || a.s[k] != b.s[k]) continue;
    ll ra = a.row, rb = b.row, on[2], os[2];
    int outer = 0;
    bool ok = true;
    for (int i = 0; i < 3; ++i) {
      if (i == k) continue;
      const bool oa = a.n[i] > 1 && a.s[i] >= a.s[k], ob = b.n[i] > 1 && b.s[i] >= b.s[k];
      if (oa || ob) {
        ok = ok && a.n[i] == b.n[i] && a.s[i] == b.s[i];
        on[outer] = a.n[i], os[outer++] = a.s[i];
      } else {
        ra += (a.n[i] - 1) * a.s[i], rb += (b.n[i] - 1) * b.s[i];
      }
    }
    if (!ok || off < ra || off + rb > a.s[k]) continue;
    const int lo = outer == 2 && os[1] < os[0];
    ll all = a.n[k] * a.s[k];
    for (int i = 0; i < outer; ++i) {
      const int o = i ^ lo;
      ok = ok && os[o] >= all;
      all = on[o] * os[o];
    }
    if (ok) return true;
  }
  return false;
}
// Whether two buffers may share a byte.
bool meet(const Rows& a, const Rows& b) {
  if (a.none() || b.none()) return false;
  const uintptr_t x = (uintptr_t)a.p, y = (uintptr_t)b.p;
  if (x + (uintptr_t)a.span() <= y || y + (uintptr_t)b.span() <= x) return false;
  return y >= x ? !beside(a, b, (ll)(y - x)) : !beside(b, a, (ll)(x - y));
}
template <int NI, int NO> bool any_meet(const Rows (&ins)[NI], const Rows (&outs)[NO]) {
  for (int i = 0; i < NO; ++i) {
    for (int j = 0; j < NI; ++j)
      if (meet(outs[i], ins[j])) return true;
    for (int j = 0; j < i; ++j)
      if (meet(outs[i], outs[j])) return true;
  }
  return false;
}

// Whether n[i] places at stride st[i] (elements), each holding what the next smaller stride spans, lie apart.
template <int N> bool rows_apart(ll row, const ll (&count)[N], const ll (&stride)[N]) {
  bool used[N] = {};
  ll span = row;
  for (int k = 0; k < N; ++k) {
    int best = -1;
    for (int i = 0; i < N; ++i)
      if (!used[i] && count[i] > 1 && (best < 0 || stride[i] < stride[best])) best = i;
    if (best < 0) return true;
    if (stride[best] < span) return false;
    span += (count[best] - 1) * stride[best];
    used[best] = true;
  }
  return true;
}
// Strides that keep every address of a buffer within 2^48 elements of its start.
template <int N> bool strides_fit(ll row, const ll (&count)[N], const ll (&stride)[N]) {
  ll span = row;
  for (int i = 0; i < N; ++i) {
    if (stride[i] < 0 || (count[i] > 1 && stride[i] > kMostElements / count[i])) return false;
    if (count[i] > 1) span += (count[i] - 1) * stride[i];
  }
  return span <= kMostElements;
}

bool conv_sizes(int B, int H, int T, int D, int W) {
  return B >= 1 && H >= 1 && T >= 0 && T <= (1 << 28) && D >= 8 && D % 8 == 0 && W >= 2 && W <= 4 && B <= (1 << 20) &&
         D <= (1 << 20) && (ll)H * D <= (1 << 20) && (ll)B * H * D <= (1LL << 31) && (ll)B * H * D * (T ? T : 1) <= kMostElements;
}
bool qk_sizes(int B, int T, int Hq, int Hqw, int Hk, int Hkw, int D) {
  return B >= 1 && T >= 0 && (ll)B * T <= (1 << 30) && Hq >= 0 && Hk >= 0 && Hq <= 32767 && Hk <= 32767 && Hq + Hk > 0 && D >= 8 &&
         D <= 256 && D % 8 == 0 && (Hq == 0 || Hqw == 1 || Hqw == Hq) && (Hk == 0 || Hkw == 1 || Hkw == Hk) &&
         (ll)B * T * (Hq > Hk ? Hq : Hk) * D <= kMostElements;
}
bool scan_sizes(int B, int H, int T, int D) {
  return B >= 1 && H >= 1 && D >= 1 && T >= 0 && T <= (1 << 28) && (ll)B * H <= (1 << 20) && (ll)B * H * D <= (1 << 26) &&
         (((ll)B * H * D + 63) / 64) * (((ll)T + KDA_GATED_SCAN_CHUNK - 1) / KDA_GATED_SCAN_CHUNK) <= (1LL << 23);
}
bool finite_f(float x) { return x >= -3.4e38f && x <= 3.4e38f; }

struct QkCall {
  const void *q, *k;
  ll qb, qt, qh, kb, kt, kh;
  const float *qw, *kw;
  int Hqw, Hkw, norm;
  float eps, scale;
  const double* freqs;
  const int* positions;
  int B, T, Hq, Hk, D, R, dtype;
};
// The checks that the forward and the adjoint share; inputs are `needed` unless nothing reads them.
int qk_check(const QkCall& c, bool needed) {
  if (c.T != 0 && needed && ((c.Hq > 0 && !c.q) || (c.Hk > 0 && !c.k))) return KDA_ERR_NULL;
  if (c.T != 0 && c.R > 0 && !c.freqs) return KDA_ERR_NULL;
  if (!valid_dtype(c.dtype)) return KDA_ERR_DTYPE;
  if (!qk_sizes(c.B, c.T, c.Hq, c.Hqw, c.Hk, c.Hkw, c.D) || c.R < 0 || c.R > c.D || c.R % 8 || c.norm < KDA_QK_NONE ||
      c.norm > KDA_QK_L2 || !(c.eps >= 0.f && finite_f(c.eps)) || !finite_f(c.scale))
    return KDA_ERR_SHAPE;
  if (c.norm == KDA_QK_NONE && (c.qw || c.kw)) return KDA_ERR_SHAPE;
  const ll nq[] = {c.B, c.T, c.Hq}, sq[] = {c.qb, c.qt, c.qh}, nk[] = {c.B, c.T, c.Hk}, sk[] = {c.kb, c.kt, c.kh};
  if ((c.Hq && !strides_fit(c.D, nq, sq)) || (c.Hk && !strides_fit(c.D, nk, sk))) return KDA_ERR_SHAPE;
  const size_t es = esize(c.dtype);
  if (!aligned(c.q, es) || !aligned(c.k, es) || !aligned(c.freqs, 8) || !aligned(c.positions, 4) || !aligned(c.qw, 4) ||
      !aligned(c.kw, 4))
    return KDA_ERR_ALIGN;
  return KDA_OK;
}
Rows qk_rows(const void* p, ll b, ll t, ll h, int B, int T, int H, int D, ll es) {
  return {p, D * es, {B, T, H}, {b * es, t * es, h * es}};
}
Rows conv_rows(const void* p, ll b, ll t, int B, int T, ll C, ll es) { return {p, C * es, {B, T, 1}, {b * es, t * es, 0}}; }
QkSideDesc side_of(const void* x, ll b, ll t, ll h, const float* w, int Hw, int H, void* y) {
  QkSideDesc d = {};
  d.x = x, d.xb = b, d.xt = t, d.xh = h, d.w = w, d.H = H, d.per_head = w && Hw > 1, d.y = y;
  return d;
}

}  // namespace
}  // namespace kda

using namespace kda;

extern "C" {

int kda_short_conv_fwd(const void* x, ll x_batch, ll x_token, const float* weight, const float* bias, const int* lengths,
                       const void* state_in, int act, void* y, void* state_out, int B, int H, int T, int D, int W,
                       int dtype, void* stream) {
  if (!weight || (T != 0 && (!x || !y))) return reject(KDA_ERR_NULL);
  if (!valid_dtype(dtype)) return reject(KDA_ERR_DTYPE);
  if (!conv_sizes(B, H, T, D, W) || (act != KDA_ACT_NONE && act != KDA_ACT_SILU)) return reject(KDA_ERR_SHAPE);
  const ll C = (ll)H * D, es = esize(dtype), n[] = {B, T}, st[] = {x_batch, x_token};
  if (!strides_fit(C, n, st)) return reject(KDA_ERR_SHAPE);
  if (!aligned(x, es) || !aligned(y, es) || !aligned(state_in, es) || !aligned(state_out, es) || !aligned(weight, 4) ||
      !aligned(bias, 4) || !aligned(lengths, 4))
    return reject(KDA_ERR_ALIGN);
  const Rows ins[] = {conv_rows(x, x_batch, x_token, B, T, C, es), flat(weight, C * W * 4), flat(bias, C * 4),
                      flat(lengths, (ll)B * 4), flat(state_in, (ll)B * (W - 1) * C * es)};
  const Rows outs[] = {flat(y, (ll)B * T * C * es), flat(state_out, (ll)B * (W - 1) * C * es)};
  if (any_meet(ins, outs)) return reject(KDA_ERR_ALIAS);
  hipStream_t s = (hipStream_t)stream;
  const hipError_t e = dtype == KDA_BF16 ? launch_conv_fwd<bf16_t>(x, x_batch, x_token, weight, bias, lengths, state_in, act, y,
                                                                   state_out, B, H, T, D, W, s)
                                         : launch_conv_fwd<float>(x, x_batch, x_token, weight, bias, lengths, state_in, act, y,
                                                                  state_out, B, H, T, D, W, s);
  return e == hipSuccess ? KDA_OK : reject(KDA_ERR_HIP);
}

int kda_short_conv_step(const void* x, ll x_batch, const float* weight, const float* bias, int act, void* state, void* y,
                        int B, int H, int D, int W, int dtype, void* stream) {
  if (!x || !weight || !state || !y) return reject(KDA_ERR_NULL);
  if (!valid_dtype(dtype)) return reject(KDA_ERR_DTYPE);
  if (!conv_sizes(B, H, 1, D, W) || (act != KDA_ACT_NONE && act != KDA_ACT_SILU)) return reject(KDA_ERR_SHAPE);
  const ll C = (ll)H * D, es = esize(dtype), n[] = {B}, st[] = {x_batch};
  if (!strides_fit(C, n, st)) return reject(KDA_ERR_SHAPE);
  if (!aligned(x, es) || !aligned(y, es) || !aligned(state, es) || !aligned(weight, 4) || !aligned(bias, 4))
    return reject(KDA_ERR_ALIGN);
  const Rows ins[] = {conv_rows(x, x_batch, 0, B, 1, C, es), flat(weight, C * W * 4), flat(bias, C * 4)};
  const Rows outs[] = {flat(y, (ll)B * C * es), flat(state, (ll)B * (W - 1) * C * es)};
  if (any_meet(ins, outs)) return reject(KDA_ERR_ALIAS);
  hipStream_t s = (hipStream_t)stream;
  const hipError_t e = dtype == KDA_BF16 ? launch_conv_step<bf16_t>(x, x_batch, weight, bias, act, state, y, B, (int)C, W, s)
                                         : launch_conv_step<float>(x, x_batch, weight, bias, act, state, y, B, (int)C, W, s);
  return e == hipSuccess ? KDA_OK : reject(KDA_ERR_HIP);
}

size_t kda_short_conv_bwd_workspace_bytes(int B, int H, int T, int D, int W, int dtype) {
  if (!valid_dtype(dtype) || !conv_sizes(B, H, T, D, W)) return 0;
  return conv_bwd_workspace_bytes(B, H, T, D, W, dtype == KDA_BF16);
}

int kda_short_conv_bwd(const void* x, ll x_batch, ll x_token, const float* weight, const float* bias, const int* lengths,
                       const void* state_in, int act, const void* dy, const float* d_state_out, void* dx, ll dx_batch,
                       ll dx_token, float* dweight, float* dbias, float* d_state_in, void* workspace,
                       size_t workspace_bytes, int B, int H, int T, int D, int W, int dtype, void* stream) {
  if (!weight || !d_state_in || (T != 0 && (!x || !dy || !dx))) return reject(KDA_ERR_NULL);
  if (!valid_dtype(dtype)) return reject(KDA_ERR_DTYPE);
  if (!conv_sizes(B, H, T, D, W) || (act != KDA_ACT_NONE && act != KDA_ACT_SILU)) return reject(KDA_ERR_SHAPE);
  const ll C = (ll)H * D, es = esize(dtype), n[] = {B, T}, st[] = {x_batch, x_token}, dst[] = {dx_batch, dx_token};
  if (!strides_fit(C, n, st) || !strides_fit(C, n, dst) || !rows_apart(C, n, dst)) return reject(KDA_ERR_SHAPE);
  if (!aligned(x, es) || !aligned(dy, es) || !aligned(dx, es) || !aligned(state_in, es) || !aligned(weight, 4) ||
      !aligned(bias, 4) || !aligned(lengths, 4) || !aligned(d_state_out, 4) || !aligned(dweight, 4) || !aligned(dbias, 4) ||
      !aligned(d_state_in, 4))
    return reject(KDA_ERR_ALIGN);
  const size_t need = dweight || dbias ? conv_bwd_workspace_bytes(B, H, T, D, W, dtype == KDA_BF16) : 0;
  if (need && (!workspace || workspace_bytes < need)) return reject(KDA_ERR_WORKSPACE);
  if (need && !aligned(workspace, 16)) return reject(KDA_ERR_ALIGN);
  const ll ns = (ll)B * (W - 1) * C;
  const Rows ins[] = {conv_rows(x, x_batch, x_token, B, T, C, es), flat(weight, C * W * 4), flat(bias, C * 4),
                      flat(lengths, (ll)B * 4), flat(state_in, ns * es), flat(dy, (ll)B * T * C * es), flat(d_state_out, ns * 4)};
  const Rows outs[] = {conv_rows(dx, dx_batch, dx_token, B, T, C, es), flat(dweight, C * W * 4), flat(dbias, C * 4),
                       flat(d_state_in, ns * 4), flat(need ? workspace : nullptr, (ll)need)};
  if (any_meet(ins, outs)) return reject(KDA_ERR_ALIAS);
  hipStream_t s = (hipStream_t)stream;
  const hipError_t e =
      dtype == KDA_BF16
          ? launch_conv_bwd<bf16_t>(x, x_batch, x_token, weight, bias, lengths, state_in, act, dy, d_state_out, dx, dx_batch,
                                    dx_token, dweight, dbias, d_state_in, workspace, B, H, T, D, W, s)
          : launch_conv_bwd<float>(x, x_batch, x_token, weight, bias, lengths, state_in, act, dy, d_state_out, dx, dx_batch,
                                   dx_token, dweight, dbias, d_state_in, workspace, B, H, T, D, W, s);
  return e == hipSuccess ? KDA_OK : reject(KDA_ERR_HIP);
}

int kda_qk_norm_rope_fwd(const void* q, ll q_batch, ll q_token, ll q_head, const void* k, ll k_batch, ll k_token, ll k_head,
                         const float* q_weight, int Hqw, const float* k_weight, int Hkw, int norm, float eps,
                         const double* freqs, const int* positions, float rope_scale, int interleaved, void* q_out,
                         void* k_out, int B, int T, int Hq, int Hk, int D, int R, int dtype, void* stream) {
  const QkCall c = {q, k, q_batch, q_token, q_head, k_batch, k_token, k_head, q_weight, k_weight, Hqw, Hkw, norm, eps,
                    rope_scale, freqs, positions, B, T, Hq, Hk, D, R, dtype};
  if (T != 0 && ((Hq > 0 && !q_out) || (Hk > 0 && !k_out))) return reject(KDA_ERR_NULL);
  const int st = qk_check(c, true);
  if (st != KDA_OK) return reject(st);
  const ll es = esize(dtype);
  if (!aligned(q_out, es) || !aligned(k_out, es)) return reject(KDA_ERR_ALIGN);
  const Rows ins[] = {qk_rows(q, q_batch, q_token, q_head, B, T, Hq, D, es), qk_rows(k, k_batch, k_token, k_head, B, T, Hk, D, es),
                      flat(q_weight, (ll)Hqw * D * 4), flat(k_weight, (ll)Hkw * D * 4), flat(freqs, (ll)R * 4),
                      flat(positions, (ll)B * T * 4)};
  const Rows outs[] = {flat(q_out, (ll)B * T * Hq * D * es), flat(k_out, (ll)B * T * Hk * D * es)};
  if (any_meet(ins, outs)) return reject(KDA_ERR_ALIAS);
  const QkSideDesc d[] = {side_of(q, q_batch, q_token, q_head, q_weight, Hqw, Hq, q_out),
                          side_of(k, k_batch, k_token, k_head, k_weight, Hkw, Hk, k_out)};
  hipStream_t s = (hipStream_t)stream;
  const hipError_t e = dtype == KDA_BF16 ? launch_qk_fwd<bf16_t>(d, freqs, positions, norm, eps, rope_scale, interleaved, B, T, D, R, s)
                                         : launch_qk_fwd<float>(d, freqs, positions, norm, eps, rope_scale, interleaved, B, T, D, R, s);
  return e == hipSuccess ? KDA_OK : reject(KDA_ERR_HIP);
}

size_t kda_qk_norm_rope_bwd_workspace_bytes(int B, int T, int Hq, int Hqw, int Hk, int Hkw, int D) {
  if (!qk_sizes(B, T, Hq, Hqw, Hk, Hkw, D)) return 0;
  return qk_bwd_workspace_bytes(B, T, Hq, Hk, D, Hqw > 1, Hkw > 1);
}

int kda_qk_norm_rope_bwd(const void* q, ll q_batch, ll q_token, ll q_head, const void* k, ll k_batch, ll k_token, ll k_head,
                         const float* q_weight, int Hqw, const float* k_weight, int Hkw, int norm, float eps,
                         const double* freqs, const int* positions, float rope_scale, int interleaved, const void* d_q,
                         const void* d_k, void* dq, ll dq_batch, ll dq_token, ll dq_head, void* dk, ll dk_batch, ll dk_token,
                         ll dk_head, float* dq_weight, float* dk_weight, void* workspace, size_t workspace_bytes, int B, int T,
                         int Hq, int Hk, int D, int R, int dtype, void* stream) {
  const QkCall c = {q, k, q_batch, q_token, q_head, k_batch, k_token, k_head, q_weight, k_weight, Hqw, Hkw, norm, eps,
                    rope_scale, freqs, positions, B, T, Hq, Hk, D, R, dtype};
  if (T != 0 && ((Hq > 0 && (!d_q || !dq)) || (Hk > 0 && (!d_k || !dk)))) return reject(KDA_ERR_NULL);
  const int st = qk_check(c, norm != KDA_QK_NONE);
  if (st != KDA_OK) return reject(st);
  if (norm == KDA_QK_NONE && (dq_weight || dk_weight)) return reject(KDA_ERR_SHAPE);
  if ((dq_weight && !Hq) || (dk_weight && !Hk)) return reject(KDA_ERR_SHAPE);
  const ll nq[] = {B, T, Hq}, sq[] = {dq_batch, dq_token, dq_head}, nk[] = {B, T, Hk}, sk[] = {dk_batch, dk_token, dk_head};
  if ((Hq && (!strides_fit(D, nq, sq) || !rows_apart(D, nq, sq))) || (Hk && (!strides_fit(D, nk, sk) || !rows_apart(D, nk, sk))))
    return reject(KDA_ERR_SHAPE);
  const ll es = esize(dtype);
  if (!aligned(d_q, es) || !aligned(d_k, es) || !aligned(dq, es) || !aligned(dk, es) || !aligned(dq_weight, 4) ||
      !aligned(dk_weight, 4))
    return reject(KDA_ERR_ALIGN);
  // a row of weights for every head where the gradient has one, whether or not weights are given
  const int qp = Hqw > 1, kp = Hkw > 1;
  const size_t need = dq_weight || dk_weight ? qk_bwd_workspace_bytes(B, T, Hq, Hk, D, qp, kp) : 0;
  if (need && (!workspace || workspace_bytes < need)) return reject(KDA_ERR_WORKSPACE);
  if (need && !aligned(workspace, 16)) return reject(KDA_ERR_ALIGN);
  const bool reads = norm != KDA_QK_NONE;
  const Rows ins[] = {qk_rows(reads ? q : nullptr, q_batch, q_token, q_head, B, T, Hq, D, es),
                      qk_rows(reads ? k : nullptr, k_batch, k_token, k_head, B, T, Hk, D, es),
                      flat(q_weight, (ll)Hqw * D * 4), flat(k_weight, (ll)Hkw * D * 4), flat(freqs, (ll)R * 4),
                      flat(positions, (ll)B * T * 4), flat(d_q, (ll)B * T * Hq * D * es), flat(d_k, (ll)B * T * Hk * D * es)};
  const Rows outs[] = {qk_rows(dq, dq_batch, dq_token, dq_head, B, T, Hq, D, es),
                       qk_rows(dk, dk_batch, dk_token, dk_head, B, T, Hk, D, es), flat(dq_weight, (ll)Hqw * D * 4),
                       flat(dk_weight, (ll)Hkw * D * 4), flat(need ? workspace : nullptr, (ll)need)};
  if (any_meet(ins, outs)) return reject(KDA_ERR_ALIAS);
  QkSideDesc d[] = {side_of(q, q_batch, q_token, q_head, q_weight, Hqw, Hq, const_cast<void*>(d_q)),
                    side_of(k, k_batch, k_token, k_head, k_weight, Hkw, Hk, const_cast<void*>(d_k))};
  d[0].dx = dq, d[0].db = dq_batch, d[0].dt = dq_token, d[0].dh = dq_head, d[0].per_head = qp;
  d[1].dx = dk, d[1].db = dk_batch, d[1].dt = dk_token, d[1].dh = dk_head, d[1].per_head = kp;
  hipStream_t s = (hipStream_t)stream;
  const hipError_t e = dtype == KDA_BF16
                           ? launch_qk_bwd<bf16_t>(d, freqs, positions, norm, eps, rope_scale, interleaved, dq_weight, dk_weight,
                                                   workspace, B, T, D, R, s)
                           : launch_qk_bwd<float>(d, freqs, positions, norm, eps, rope_scale, interleaved, dq_weight, dk_weight,
                                                  workspace, B, T, D, R, s);
  return e == hipSuccess ? KDA_OK : reject(KDA_ERR_HIP);
}

int kda_rope_frequencies(double* freqs, double* rope_scale, int R, double base, int scaling, double factor,
                         double trained_length, double fast_turns, double slow_turns) {
  if (!freqs || !rope_scale) return reject(KDA_ERR_NULL);
  const double most = 1e300;
  if (R <= 0 || R % 2 || R > (1 << 20) || !(base > 1 && base < most) || scaling < KDA_ROPE_PLAIN || scaling > KDA_ROPE_PARTS ||
      !(factor >= 1 && factor < most) || (scaling == KDA_ROPE_BASE && R <= 2))
    return reject(KDA_ERR_SHAPE);
  if (scaling == KDA_ROPE_PARTS &&
      !(trained_length > 0 && trained_length < most && slow_turns > 0 && fast_turns > slow_turns && fast_turns < most))
    return reject(KDA_ERR_SHAPE);
  const int n = R / 2;
  if (scaling == KDA_ROPE_BASE) base *= pow(factor, (double)R / (R - 2));
  if (!(base < 1e308)) return reject(KDA_ERR_SHAPE);
  // the pair (not a whole number) that turns `turns` times over the trained length
  const auto pair_of = [=](double turns) { return R * log(trained_length / (turns * 2 * M_PI)) / (2 * log(base)); };
  const double lo = scaling == KDA_ROPE_PARTS ? fmax(floor(pair_of(fast_turns)), 0) : 0;
  // (the first pair behind the ramp may stand behind the table, whose last pair is n - 1: a cut there would steepen the ramp)
  const double hi = scaling == KDA_ROPE_PARTS ? fmin(ceil(pair_of(slow_turns)), R - 1) : 0;
  for (int p = 0; p < n; ++p) {
    double f = pow(base, -2.0 * p / R);
    if (scaling == KDA_ROPE_LINEAR) f /= factor;
    if (scaling == KDA_ROPE_PARTS) {
      const double share = fmin(fmax((p - lo) / fmax(hi - lo, 0.001), 0), 1);
      f = f * (1 - share) + f / factor * share;
    }
    freqs[p] = f;
  }
  *rope_scale = scaling == KDA_ROPE_PARTS ? 0.1 * log(factor) + 1 : 1;
  return KDA_OK;
}

size_t kda_gated_scan_workspace_bytes(int B, int H, int T, int D, int dtype) {
  if (!valid_dtype(dtype) || !scan_sizes(B, H, T, D)) return 0;
  return scan_workspace_bytes(B, H, T, D, dtype == KDA_BF16);
}

int kda_gated_scan_fwd(const void* x, const void* z, const float* A_log, const float* dt_bias, const void* input_gate,
                       const int* lengths, const float* state_in, int normalize, void* y, float* state_out, float* ckpt,
                       void* workspace, size_t workspace_bytes, int B, int H, int T, int D, int dtype, void* stream) {
  if (!A_log || (T != 0 && (!x || !z || !y))) return reject(KDA_ERR_NULL);
  if (!valid_dtype(dtype)) return reject(KDA_ERR_DTYPE);
  if (!scan_sizes(B, H, T, D)) return reject(KDA_ERR_SHAPE);
  const ll es = esize(dtype), n = (ll)B * H * T * D * es, ns = (ll)B * H * D * 4, hd = (ll)H * D * 4;
  if (!aligned(x, es) || !aligned(z, es) || !aligned(input_gate, es) || !aligned(y, es) || !aligned(A_log, 4) ||
      !aligned(dt_bias, 4) || !aligned(lengths, 4) || !aligned(state_in, 4) || !aligned(state_out, 4) || !aligned(ckpt, 4))
    return reject(KDA_ERR_ALIGN);
  const size_t need = scan_workspace_bytes(B, H, T, D, dtype == KDA_BF16);
  if (need && (!workspace || workspace_bytes < need)) return reject(KDA_ERR_WORKSPACE);
  if (need && !aligned(workspace, 256)) return reject(KDA_ERR_ALIGN);
  const Rows ins[] = {flat(x, n), flat(z, n), flat(input_gate, n), flat(A_log, (ll)H * 4), flat(dt_bias, hd),
                      flat(lengths, (ll)B * 4), flat(state_in == state_out ? nullptr : state_in, ns)};
  const ll nc = (T + KDA_GATED_SCAN_CHUNK - 1) / KDA_GATED_SCAN_CHUNK * ns;
  const Rows outs[] = {flat(y, n), flat(state_out, ns), flat(ckpt, nc), flat(need ? workspace : nullptr, (ll)need)};
  if (any_meet(ins, outs)) return reject(KDA_ERR_ALIAS);
  hipStream_t s = (hipStream_t)stream;
  const hipError_t e = dtype == KDA_BF16 ? launch_scan_fwd<bf16_t>(x, z, A_log, dt_bias, input_gate, lengths, state_in, normalize, y,
                                                                   state_out, ckpt, workspace, B, H, T, D, s)
                                         : launch_scan_fwd<float>(x, z, A_log, dt_bias, input_gate, lengths, state_in, normalize, y,
                                                                  state_out, ckpt, workspace, B, H, T, D, s);
  if (e != hipSuccess) return reject(KDA_ERR_HIP);
  count_call(KDA_COUNTER_CHUNK_FWD);
  return KDA_OK;
}

int kda_gated_scan_step(const void* x, const void* z, const float* A_log, const float* dt_bias, const void* input_gate,
                        int normalize, float* state, void* y, int B, int H, int D, int dtype, void* stream) {
  if (!x || !z || !A_log || !state || !y) return reject(KDA_ERR_NULL);
  if (!valid_dtype(dtype)) return reject(KDA_ERR_DTYPE);
  if (!scan_sizes(B, H, 1, D)) return reject(KDA_ERR_SHAPE);
  const ll es = esize(dtype), n = (ll)B * H * D * es, ns = (ll)B * H * D * 4, hd = (ll)H * D * 4;
  if (!aligned(x, es) || !aligned(z, es) || !aligned(input_gate, es) || !aligned(y, es) || !aligned(A_log, 4) ||
      !aligned(dt_bias, 4) || !aligned(state, 4))
    return reject(KDA_ERR_ALIGN);
  const Rows ins[] = {flat(x, n), flat(z, n), flat(input_gate, n), flat(A_log, (ll)H * 4), flat(dt_bias, hd)};
  const Rows outs[] = {flat(y, n), flat(state, ns)};
  if (any_meet(ins, outs)) return reject(KDA_ERR_ALIAS);
  hipStream_t s = (hipStream_t)stream;
  const hipError_t e = dtype == KDA_BF16 ? launch_scan_step<bf16_t>(x, z, A_log, dt_bias, input_gate, normalize, state, y, B, H, D, s)
                                         : launch_scan_step<float>(x, z, A_log, dt_bias, input_gate, normalize, state, y, B, H, D, s);
  if (e != hipSuccess) return reject(KDA_ERR_HIP);
  count_call(KDA_COUNTER_RECURRENT_STEP);
  return KDA_OK;
}

size_t kda_gated_scan_bwd_workspace_bytes(int B, int H, int T, int D, int dtype) {
  if (!valid_dtype(dtype) || !scan_sizes(B, H, T, D)) return 0;
  return scan_bwd_workspace_bytes(B, H, T, D, dtype == KDA_BF16);
}

int kda_gated_scan_bwd(const void* x, const void* z, const float* A_log, const float* dt_bias, const void* input_gate,
                       const int* lengths, int normalize, const float* ckpt, const void* dy, const float* d_state_out,
                       void* dx, void* dz, void* d_input_gate, float* dA_log, float* d_dt_bias, float* d_state_in,
                       void* workspace, size_t workspace_bytes, int B, int H, int T, int D, int dtype, void* stream) {
  if (!A_log || !d_state_in || (T != 0 && (!x || !z || !ckpt || !dy || !dx || !dz))) return reject(KDA_ERR_NULL);
  if (T != 0 && (input_gate != nullptr) != (d_input_gate != nullptr)) return reject(KDA_ERR_NULL);
  if (!valid_dtype(dtype)) return reject(KDA_ERR_DTYPE);
  if (!scan_sizes(B, H, T, D)) return reject(KDA_ERR_SHAPE);
  const ll es = esize(dtype), n = (ll)B * H * T * D * es, ns = (ll)B * H * D * 4, hd = (ll)H * D * 4;
  if (!aligned(x, es) || !aligned(z, es) || !aligned(input_gate, es) || !aligned(dy, es) || !aligned(dx, es) || !aligned(dz, es) ||
      !aligned(d_input_gate, es) || !aligned(A_log, 4) || !aligned(dt_bias, 4) || !aligned(lengths, 4) || !aligned(ckpt, 4) ||
      !aligned(d_state_out, 4) || !aligned(dA_log, 4) || !aligned(d_dt_bias, 4) || !aligned(d_state_in, 4))
    return reject(KDA_ERR_ALIGN);
  const size_t need = scan_bwd_workspace_bytes(B, H, T, D, dtype == KDA_BF16);
  if (need && (!workspace || workspace_bytes < need)) return reject(KDA_ERR_WORKSPACE);
  if (need && !aligned(workspace, 256)) return reject(KDA_ERR_ALIGN);
  const ll nc = (T + KDA_GATED_SCAN_CHUNK - 1) / KDA_GATED_SCAN_CHUNK * ns;
  const Rows ins[] = {flat(x, n), flat(z, n), flat(input_gate, n), flat(A_log, (ll)H * 4), flat(dt_bias, hd),
                      flat(lengths, (ll)B * 4), flat(ckpt, nc), flat(dy, n), flat(d_state_out, ns)};
  const Rows outs[] = {flat(dx, n), flat(dz, n), flat(d_input_gate, n), flat(dA_log, (ll)H * 4), flat(d_dt_bias, hd),
                       flat(d_state_in, ns), flat(need ? workspace : nullptr, (ll)need)};
  if (any_meet(ins, outs)) return reject(KDA_ERR_ALIAS);
  hipStream_t s = (hipStream_t)stream;
  const hipError_t e =
      dtype == KDA_BF16 ? launch_scan_bwd<bf16_t>(x, z, A_log, dt_bias, input_gate, lengths, normalize, ckpt, dy, d_state_out, dx, dz,
                                                  d_input_gate, dA_log, d_dt_bias, d_state_in, workspace, B, H, T, D, s)
                        : launch_scan_bwd<float>(x, z, A_log, dt_bias, input_gate, lengths, normalize, ckpt, dy, d_state_out, dx, dz,
                                                 d_input_gate, dA_log, d_dt_bias, d_state_in, workspace, B, H, T, D, s);
  if (e != hipSuccess) return reject(KDA_ERR_HIP);
  count_call(KDA_COUNTER_CHUNK_BWD);
  return KDA_OK;
}

}  // extern "C"
