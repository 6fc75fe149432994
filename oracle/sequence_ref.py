"""Float64 numpy definitions of the operators between a layer's projections and its mixer: short causal convolution,
norm of queries and keys with their rotation, gated linear recurrence (token by token), and their adjoints.  Nothing here
is shared with the GPU path.
"""
import numpy as np


def _f64(*xs):
    return tuple(None if x is None else np.asarray(x, np.float64) for x in xs)


def _lens(lengths, B, T):
    return [T] * B if lengths is None else [min(max(int(n), 0), T) for n in lengths]


def _sigmoid(x):
    return 1.0 / (1.0 + np.exp(-x))


# ------------------------------------------------------------------ short convolution
def _conv_pre(x, w, bias, state):
    """(the inputs behind the kept ones (B, W-1+T, C), pre-activations (B,T,C))."""
    B, T, C = x.shape
    W = w.shape[-1]
    full = np.concatenate((np.zeros((B, W - 1, C)) if state is None else state, x), 1)
    pre = np.zeros((B, T, C)) + (0.0 if bias is None else bias)
    for j in range(W):
        pre = pre + full[:, j:j + T] * w[:, j]
    return full, pre


def short_conv(x, w, bias=None, state=None, lengths=None, silu=True, heads=1):
    """(y (B,heads,T,C/heads), state_out (B,W-1,C)); rows of y behind a length are 0."""
    x, w, bias, state = _f64(x, w, bias, state)
    B, T, C = x.shape
    W = w.shape[-1]
    full, pre = _conv_pre(x, w, bias, state)
    y = pre * _sigmoid(pre) if silu else pre.copy()
    end = np.empty((B, W - 1, C))
    for b, n in enumerate(_lens(lengths, B, T)):
        y[b, n:] = 0
        end[b] = full[b, n:n + W - 1]
    return y.reshape(B, T, heads, C // heads).transpose(0, 2, 1, 3), end


def short_conv_adjoint(x, w, bias, state, dy, d_state=None, lengths=None, silu=True):
    x, w, bias, state, dy = _f64(x, w, bias, state, dy)
    B, T, C = x.shape
    W = w.shape[-1]
    full, pre = _conv_pre(x, w, bias, state)
    d = dy.transpose(0, 2, 1, 3).reshape(B, T, C)
    if silu:
        s = _sigmoid(pre)
        d = d * (s + pre * s * (1 - s))
    d = d.copy()
    dfull = np.zeros_like(full)
    for b, n in enumerate(_lens(lengths, B, T)):
        d[b, n:] = 0
        if d_state is not None:
            dfull[b, n:n + W - 1] += d_state[b]
    dw = np.zeros_like(w)
    for j in range(W):
        dfull[:, j:j + T] += d * w[:, j]
        # (inputs behind a sequence's end meet zero cotangents; they may hold anything)
        dw[:, j] = np.where(d != 0, d * full[:, j:j + T], 0.0).sum((0, 1))
    return {"dx": dfull[:, W - 1:], "dstate_in": dfull[:, :W - 1], "dweight": dw, "dbias": d.sum((0, 1))}


# ------------------------------------------------------------------ norm and rotation
def rope_frequencies(R, base=10000.0, scaling=None, factor=1.0, trained=4096.0, fast=32.0, slow=1.0):
    """([radians per token], scale): the definitions written out pair by pair."""
    if scaling == "base":
        base = base * factor ** (R / (R - 2.0))
    out = []
    for p in range(R // 2):
        f = base ** (-2.0 * p / R)
        if scaling == "linear":
            f = f / factor
        if scaling == "parts":
            # the pair that turns n times: base^(-2 p / R) trained = 2 pi n
            first = max(np.floor(R / 2.0 * np.log(trained / (2 * np.pi * fast)) / np.log(base)), 0.0)
            last = min(np.ceil(R / 2.0 * np.log(trained / (2 * np.pi * slow)) / np.log(base)), R - 1.0)
            share = min(max((p - first) / max(last - first, 1e-3), 0.0), 1.0)
            f = (1 - share) * f + share * f / factor
        out.append(f)
    return np.array(out), (0.1 * np.log(factor) + 1.0 if scaling == "parts" else 1.0)


def _turn(x, angle, scale, interleaved):
    """x (..., D) with the first 2 * angle.shape[-1] channels turned by `angle`."""
    y, n = x.copy(), angle.shape[-1]
    a = np.arange(0, 2 * n, 2) if interleaved else np.arange(n)
    b = a + 1 if interleaved else a + n
    c, s = np.cos(angle) * scale, np.sin(angle) * scale
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def _qk_rows(x, norm, eps):
    D = x.shape[-1]
    if norm is None:
        return np.ones(x.shape[:-1] + (1,))
    ss = (x * x).sum(-1, keepdims=True) / (D if norm == "rms" else 1)
    with np.errstate(divide="ignore"):
        return 1.0 / np.sqrt(ss + eps)


def qk_norm_rope(x, weight, freqs, positions=None, norm="rms", eps=1e-6, interleaved=False, rope_scale=1.0):
    """x (B,T,H,D) -> (B,H,T,D)."""
    x, weight, freqs = _f64(x, weight, freqs)
    B, T, H, D = x.shape
    pos = np.broadcast_to(np.arange(T), (B, T)) if positions is None else np.asarray(positions, np.float64)
    angle = pos[:, :, None, None] * (np.zeros(0) if freqs is None else freqs)
    xn = x * _qk_rows(x, norm, eps)
    if weight is not None:
        xn = xn * weight
    return _turn(xn, angle, rope_scale, interleaved).transpose(0, 2, 1, 3)


def qk_norm_rope_adjoint(x, weight, freqs, dy, positions=None, norm="rms", eps=1e-6, interleaved=False, rope_scale=1.0):
    """(dx (B,T,H,D), dweight in weight's shape or None)."""
    x, weight, freqs, dy = _f64(x, weight, freqs, dy)
    B, T, H, D = x.shape
    pos = np.broadcast_to(np.arange(T), (B, T)) if positions is None else np.asarray(positions, np.float64)
    angle = pos[:, :, None, None] * (np.zeros(0) if freqs is None else freqs)
    p = _turn(dy.transpose(0, 2, 1, 3), -angle, rope_scale, interleaved)
    r = _qk_rows(x, norm, eps)
    xh = x * r
    dw = None
    if weight is not None:
        dw = (p * xh).sum((0, 1))
        dw = dw.sum(0, keepdims=True) if weight.shape[0] == 1 else dw
        p = p * weight
    if norm is None:
        return p, dw
    dot = (p * xh).sum(-1, keepdims=True) / (D if norm == "rms" else 1)
    return r * (p - xh * dot), dw


# ------------------------------------------------------------------ gated recurrence
def scan_gates(z, A_log, dt_bias, normalize):
    """(g, a, n, dg/dz) of z (B,H,...,D)."""
    z, A_log, dt_bias = _f64(z, A_log, dt_bias)
    H, D = z.shape[1], z.shape[-1]
    mid = (1,) * (z.ndim - 3)
    t = z + (0.0 if dt_bias is None else dt_bias.reshape((1, H) + mid + (D,)))
    m = np.exp(np.clip(A_log, -10, 20)).reshape((1, H) + mid + (1,))
    g = -m * np.logaddexp(t, 0.0)
    n = np.sqrt(-np.expm1(2 * g)) if normalize else np.ones_like(g)
    return g, np.exp(g), n, -m * _sigmoid(t)


def gated_scan(x, z, A_log, dt_bias=None, state=None, gate=None, lengths=None, normalize=True):
    """(y (B,H,T,D), state_out (B,H,D), states before every token (B,H,T,D)); rows of y behind a length are 0."""
    x, gate, state = _f64(x, gate, state)
    B, H, T, D = x.shape
    _, a, n, _ = scan_gates(z, A_log, dt_bias, normalize)
    u = x * n * (1.0 if gate is None else _sigmoid(gate))
    h = np.zeros((B, H, D)) if state is None else state.copy()
    y, before = np.zeros((B, H, T, D)), np.zeros((B, H, T, D))
    for b, k in enumerate(_lens(lengths, B, T)):
        for t in range(T):
            before[b, :, t] = h[b]
            if t < k:
                h[b] = a[b, :, t] * h[b] + u[b, :, t]
                y[b, :, t] = h[b]
    return y, h, before


def gated_scan_adjoint(x, z, A_log, dt_bias, state, dy, d_state=None, gate=None, lengths=None, normalize=True):
    x, gate, dy = _f64(x, gate, dy)
    B, H, T, D = x.shape
    g, a, n, slope = scan_gates(z, A_log, dt_bias, normalize)
    s = np.ones_like(x) if gate is None else _sigmoid(gate)
    _, _, before = gated_scan(x, z, A_log, dt_bias, state, gate, lengths, normalize)
    r = np.zeros((B, H, D)) if d_state is None else np.array(d_state, np.float64)
    R = np.zeros((B, H, T, D))
    for b, k in enumerate(_lens(lengths, B, T)):
        for t in reversed(range(k)):
            R[b, :, t] = r[b] + dy[b, :, t]
            r[b] = a[b, :, t] * R[b, :, t]
    dg = R * a * before
    if normalize:
        with np.errstate(divide="ignore", invalid="ignore"):
            dg = dg - np.where(n > 0, R * s * x * a * a / n, 0.0)
    dz = dg * slope
    inside = (np.asarray(A_log, np.float64) >= -10) & (np.asarray(A_log, np.float64) <= 20)
    out = {"dx": R * n * s, "dz": dz, "dA_log": (dg * g).sum((0, 2, 3)) * inside, "ddt_bias": dz.sum((0, 2)),
           "dstate_in": r, "R": R, "before": before}
    if gate is not None:
        out["dinput_gate"] = R * n * x * s * (1 - s)
    return out
