"""Float64 numpy definitions of the operators beside the delta rule: attention with a constant decay per
head (token by token) and its adjoint, layer norm and its adjoint, and the 8-bit form of activations.
Nothing here is shared with the GPU path.
"""
import numpy as np


def _lens(lengths, B, T):
    return [T] * B if lengths is None else [min(max(int(n), 0), T) for n in lengths]


def decay_attn(q, k, v, log_decay, state_in=None, lengths=None, scale=None):
    """S_t = e^g S + k_t v_t^T, o_t = scale S_t^T q_t.  Returns (o, S); rows of o behind a length are 0."""
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    B, H, T, K = q.shape
    V = v.shape[-1]
    scale = K ** -0.5 if scale is None else scale
    a = np.exp(np.asarray(log_decay, np.float64))
    S = np.zeros((B, H, K, V)) if state_in is None else np.array(state_in, np.float64)
    o = np.zeros((B, H, T, V))
    for b, n in enumerate(_lens(lengths, B, T)):
        for t in range(n):
            S[b] = a[:, None, None] * S[b] + k[b, :, t, :, None] * v[b, :, t, None, :]
            o[b, :, t] = scale * np.einsum("hk,hkv->hv", q[b, :, t], S[b])
    return o, S


def decay_attn_adjoint(q, k, v, log_decay, state_in, d_o, d_state_out=None, lengths=None, scale=None):
    """Gradients of sum(o d_o) + sum(S_T d_state_out): dict(dq, dk, dv, dstate_in)."""
    q, k, v, d_o = (np.asarray(x, np.float64) for x in (q, k, v, d_o))
    B, H, T, K = q.shape
    V = v.shape[-1]
    scale = K ** -0.5 if scale is None else scale
    a = np.exp(np.asarray(log_decay, np.float64))[:, None, None]
    S = np.zeros((B, H, K, V)) if state_in is None else np.array(state_in, np.float64)
    R = np.zeros((B, H, K, V)) if d_state_out is None else np.array(d_state_out, np.float64)
    dq, dk, dv = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)
    for b, n in enumerate(_lens(lengths, B, T)):
        for t in range(n):
            S[b] = a * S[b] + k[b, :, t, :, None] * v[b, :, t, None, :]
            dq[b, :, t] = scale * np.einsum("hkv,hv->hk", S[b], d_o[b, :, t])
        for t in reversed(range(n)):
            R[b] += scale * q[b, :, t, :, None] * d_o[b, :, t, None, :]
            dk[b, :, t] = np.einsum("hkv,hv->hk", R[b], v[b, :, t])
            dv[b, :, t] = np.einsum("hkv,hk->hv", R[b], k[b, :, t])
            R[b] = a * R[b]
    return {"dq": dq, "dk": dk, "dv": dv, "dstate_in": R}


def layer_norm(x, weight=None, bias=None, eps=1e-5):
    """(y, mean, rstd) over the last axis of (B,H,T,D); weight and bias (H,D)."""
    x = np.asarray(x, np.float64)
    mean = x.mean(-1)
    rstd = 1.0 / np.sqrt(((x - mean[..., None]) ** 2).mean(-1) + eps)
    y = (x - mean[..., None]) * rstd[..., None]
    if weight is not None:
        y = y * np.asarray(weight, np.float64)[None, :, None]
    if bias is not None:
        y = y + np.asarray(bias, np.float64)[None, :, None]
    return y, mean, rstd


def layer_norm_adjoint(x, weight, mean, rstd, dy):
    """(dx, dweight, dbias) from the given statistics."""
    x, dy, rstd = (np.asarray(a, np.float64) for a in (x, dy, rstd))
    xh = (x - np.asarray(mean, np.float64)[..., None]) * rstd[..., None]
    p = dy if weight is None else dy * np.asarray(weight, np.float64)[None, :, None]
    dx = rstd[..., None] * (p - p.mean(-1, keepdims=True) - xh * (p * xh).mean(-1, keepdims=True))
    return dx, (dy * xh).sum((0, 2)), dy.sum((0, 2))


def e4m3_values():
    """The value of every e4m3 code (OCP: bias 7, no infinity, S.1111.111 = NaN)."""
    out = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        mag = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        out[c] = np.nan if (c & 127) == 127 else (-mag if c >= 128 else mag)
    return out


def ckpt_pack(x):
    """(codes, scales) of float32-representable x (rows, D), by the definition: the smallest e >= -127 with
    amax <= 448 * 2^e per group, the nearest e4m3 value of x / 2^e, ties to the even code."""
    x = np.asarray(x, np.float64)
    rows, D = x.shape
    G = min(D, 32)
    xg = x.reshape(rows, D // G, G)
    fin = np.isfinite(xg)
    amax = np.where(fin, np.abs(xg), 0.0).max(-1)
    e = np.full(amax.shape, -127)
    while True:
        low = amax > 448.0 * 2.0 ** e
        if not low.any():
            break
        e = e + low
    y = np.where(fin, xg, 0.0) / 2.0 ** e[..., None]
    pos = e4m3_values()[:127]                                 # 0 .. 448, ascending
    mag = np.abs(y)
    hi = np.searchsorted(pos, mag).clip(0, 126)
    lo = (hi - 1).clip(0)
    dl, dh = mag - pos[lo], pos[hi] - mag
    code = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    code = code | (np.signbit(xg) * 128)
    code = np.where(fin, code, 127)
    return code.reshape(rows, D).astype(np.uint8), (e + 127).astype(np.uint8)


def ckpt_unpack(codes, scales):
    D, n = codes.shape[-1], scales.shape[-1]
    return e4m3_values()[codes] * np.repeat(2.0 ** (scales.astype(np.float64) - 127), D // n, -1)
