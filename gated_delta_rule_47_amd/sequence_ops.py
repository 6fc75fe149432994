"""Operators between a layer's projections and its mixer, and the recurrence without a matrix state: short causal
convolution, norm of queries and keys with the rotation by their positions, gated linear recurrence; each with its
adjoint, the convolution and the recurrence with their single-token forms.

Argument marshalling only, as in layer_ops.  Projections are (B, T, channels) with any strides of batch and token
(slices of a wider projection), heads (B, H, T, D) and contiguous.  Every tensor of a call lives on one GPU; the call
runs on that GPU's current stream whatever the current device is.
"""
from __future__ import annotations

import ctypes

import torch

from . import _lib, KdaError
from .layer_ops import _F32, _I32, _U8, _bytes, _code, _gpu, _opt, _ptr, _refuse

__all__ = ["short_conv_fwd", "short_conv_step", "short_conv_bwd_workspace_bytes", "short_conv_bwd", "qk_norm_rope_fwd",
           "qk_norm_rope_bwd_workspace_bytes", "qk_norm_rope_bwd", "rope_frequencies", "GATED_SCAN_CHUNK",
           "gated_scan_workspace_bytes", "gated_scan_fwd", "gated_scan_step", "gated_scan_bwd_workspace_bytes",
           "gated_scan_bwd"]

_F64 = torch.float64
GATED_SCAN_CHUNK = 32                       # KDA_GATED_SCAN_CHUNK
_ACTS = {None: 0, "silu": 1}
_NORMS = {None: 0, "rms": 1, "l2": 2}
_SCALINGS = {None: 0, "linear": 1, "base": 2, "parts": 3}


def _one_of(name, value, table):
    try:
        return table[value]
    except (KeyError, TypeError):
        raise ValueError("%s must be one of %s, got %r" % (name, ", ".join(repr(k) for k in table), value)) from None


def _strided(name, t, shape, dtype, dev):
    """(address, strides) of a tensor of this shape whose last axis is dense; the other strides are the caller's."""
    try:
        st = t.stride()
        if t.shape == shape and t.dtype is dtype and t.get_device() == dev and (st[-1] == 1 or shape[-1] == 1 or not t.numel()):
            return t.data_ptr(), st
    except AttributeError:
        pass
    if isinstance(t, torch.Tensor) and tuple(t.shape) == tuple(shape) and t.dtype == dtype and t.get_device() == dev:
        raise ValueError("%s must have its channels next to each other" % name)
    _refuse(name, t, shape, dtype, dev)


_INT = 0x7fffffff


def _fits(fn, *sizes):
    """Sizes are handed over in 32 bits: what has more is refused here, as the library refuses what is too large for it."""
    if max(sizes) > _INT:
        raise KdaError(fn, _lib.KDA_ERR_SHAPE)


def _need(fn, *sizes):
    _fits(fn, *sizes)
    return _bytes(fn, *sizes)


_entries = {}


def _run(dev, fn, *args):
    """The call on GPU dev's current stream, with dev current while it launches."""
    f = _entries.get(fn)
    if f is None:
        f = _entries[fn] = getattr(_lib.load(), fn)
    c = torch._C
    if dev == c._cuda_getDevice():
        st = f(*args, c._cuda_getCurrentRawStream(dev))
    else:
        with torch.cuda.device(dev):
            st = f(*args, c._cuda_getCurrentRawStream(dev))
    if st:
        raise KdaError(fn, st)


def _workspace(workspace, need, like):
    """(tensor kept alive, address, bytes): the caller's, or `need` bytes from torch's caching allocator."""
    if workspace is None:
        if not need:
            return None, None, 0
        workspace = like.new_empty(need, dtype=_U8)
        return workspace, workspace.data_ptr(), need
    if workspace.get_device() != like.get_device() or not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous and on the call's GPU")
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


def short_conv_fwd(x, weight, bias=None, state_in=None, lengths=None, activation="silu", heads=1, output_state=True,
                   out=None, state_out=None):
    """Causal depthwise convolution y_t = act(bias + sum_j weight[:, j] x_{t-W+1+j}) of a projection x (B,T,C), weight
    (C,W) float32 with W in 2..4, bias (C,) float32, activation "silu" or None.  Returns (y, state_out): y
    (B,heads,T,C/heads), state_out (B,W-1,C) the last inputs of every sequence (None when output_state is False), to be
    the next call's state_in or short_conv_step's state.  state_in None means zeros.  lengths (B,) int32 ends each
    sequence early: y's rows behind it are left as they are in `out` (uninitialised without one)."""
    B, T, C = x.shape
    W = weight.shape[-1]
    dt, dev = x.dtype, x.get_device()
    code, act = _code(dt), _one_of("activation", activation, _ACTS)
    if not 0 < x.numel() <= _INT or W > 4:
        _fits("kda_short_conv_fwd", B, T, C, W)
    if heads < 1 or C % heads:
        raise ValueError("%d channels do not make %r heads" % (C, heads))
    shape, state = (B, heads, T, C // heads), (B, W - 1, C)
    px, sx = _strided("x", x, (B, T, C), dt, dev)
    pw, pb = _ptr("weight", weight, (C, W), _F32, dev), _opt("bias", bias, (C,), _F32, dev)
    pn, ps = _opt("lengths", lengths, (B,), _I32, dev), _opt("state_in", state_in, state, dt, dev)
    po, pe = _opt("out", out, shape, dt, dev), _opt("state_out", state_out, state, dt, dev)
    _gpu(dev)
    if out is None:
        out = x.new_empty(shape)
        po = out.data_ptr()
    if not output_state:
        state_out = pe = None
    elif state_out is None:
        state_out = x.new_empty(state)
        pe = state_out.data_ptr()
    _run(dev, "kda_short_conv_fwd", px, sx[0], sx[1], pw, pb, pn, ps, act, po, pe, B, heads, T, C // heads, W,
         code)
    return out, state_out


def short_conv_step(x, weight, bias, state, activation="silu", out=None):
    """One token of short_conv_fwd: x (B,C); state (B,W-1,C) in x's dtype is updated in place.  Returns y (B,C)."""
    B, C = x.shape
    W = weight.shape[-1]
    dt, dev = x.dtype, x.get_device()
    code, act = _code(dt), _one_of("activation", activation, _ACTS)
    if not 0 < x.numel() <= _INT or W > 4:
        _fits("kda_short_conv_step", B, C, W)
    px, sx = _strided("x", x, (B, C), dt, dev)
    pw, pb = _ptr("weight", weight, (C, W), _F32, dev), _opt("bias", bias, (C,), _F32, dev)
    ps = _ptr("state", state, (B, W - 1, C), dt, dev)
    po = None if out is None else _ptr("out", out, (B, C), dt, dev)
    if dev < 0:
        _gpu(dev)
    if po is None:
        out = torch.empty_like(x) if sx[0] == C else x.new_empty((B, C))
        po = out.data_ptr()
    _run(dev, "kda_short_conv_step", px, sx[0], pw, pb, act, ps, po, B, 1, C, W, code)
    return out


def short_conv_bwd_workspace_bytes(B, H, T, D, W, dtype=torch.bfloat16) -> int:
    return _need("kda_short_conv_bwd_workspace_bytes", B, H, T, D, W, _code(dtype))


def short_conv_bwd(x, weight, bias, state_in, dy, d_state_out=None, lengths=None, activation="silu", want_params=True,
                   dx_out=None, workspace=None):
    """Gradients of sum(y * dy) + sum(state_out * d_state_out): dict(dx, dweight, dbias, dstate_in), dx (B,T,C) in dy's
    dtype (into dx_out, which may be a slice of a wider gradient), the rest float32 (dweight and dbias None without
    want_params).  dy (B,H,T,C/H).  Rows of dx behind a sequence's length are zero."""
    B, T, C = x.shape
    W = weight.shape[-1]
    dt, dev = x.dtype, x.get_device()
    code, act = _code(dt), _one_of("activation", activation, _ACTS)
    if not 0 < x.numel() <= _INT or W > 4:
        _fits("kda_short_conv_bwd", B, T, C, W)
    H = dy.shape[1]
    if H < 1 or C % H:
        raise ValueError("%d channels do not make %d heads" % (C, H))
    px, sx = _strided("x", x, (B, T, C), dt, dev)
    pw, pb = _ptr("weight", weight, (C, W), _F32, dev), _opt("bias", bias, (C,), _F32, dev)
    pn, ps = _opt("lengths", lengths, (B,), _I32, dev), _opt("state_in", state_in, (B, W - 1, C), dt, dev)
    pd = _ptr("dy", dy, (B, H, T, C // H), dt, dev)
    pe = _opt("d_state_out", d_state_out, (B, W - 1, C), _F32, dev)
    if dx_out is None:
        dx_out = x.new_empty((B, T, C))
    pdx, sdx = _strided("dx_out", dx_out, (B, T, C), dt, dev)
    _gpu(dev)
    d0 = weight.new_empty((B, W - 1, C))
    dw = db = pdw = pdb = None
    need = 0
    if want_params:
        dw, db = torch.empty_like(weight), weight.new_empty((C,))
        pdw, pdb = dw.data_ptr(), db.data_ptr()
        need = _bytes("kda_short_conv_bwd_workspace_bytes", B, H, T, C // H, W, code)
    ws, pws, nws = _workspace(workspace, need, weight)
    _run(dev, "kda_short_conv_bwd", px, sx[0], sx[1], pw, pb, pn, ps, act, pd, pe, pdx, sdx[0], sdx[1], pdw, pdb, d0.data_ptr(), pws, nws, B, H, T, C // H, W, code)
    return dict(dx=dx_out, dweight=dw, dbias=db, dstate_in=d0)


def rope_frequencies(rot_dim, base=10000.0, scaling=None, factor=1.0, trained_length=4096, fast_turns=32.0,
                     slow_turns=1.0, device=None):
    """(freqs, rope_scale) for qk_norm_rope_fwd: radians per token of the rot_dim / 2 pairs, float64, and the scale of
    the rotated channels.  scaling None: base^(-2p / rot_dim); "linear": slowed by factor; "base": the base raised so
    that the slowest pair is slowed by factor; "parts": pairs of more than fast_turns turns over trained_length tokens
    left, those below slow_turns slowed by factor, shares between, rope_scale = 0.1 ln(factor) + 1."""
    n = max(int(rot_dim) // 2, 1)
    if n > 1 << 19:                            # (the library's limit, before the table is made)
        raise KdaError("kda_rope_frequencies", _lib.KDA_ERR_SHAPE)
    table, scale = (ctypes.c_double * n)(), ctypes.c_double()
    st = _lib.load().kda_rope_frequencies(table, ctypes.byref(scale), int(rot_dim), float(base),
                                          _one_of("scaling", scaling, _SCALINGS), float(factor), float(trained_length),
                                          float(fast_turns), float(slow_turns))
    if st != _lib.KDA_OK:
        raise KdaError("kda_rope_frequencies", st)
    return torch.tensor(list(table), dtype=_F64, device=device), scale.value


def _side(name, x, B, T, D, weight, dt, dev):
    """(heads, rows of weights, address of x, its strides, address of weights) of the queries or the keys; x may be None."""
    if x is None:
        if weight is not None:
            raise ValueError("%s_weight without %s" % (name, name))
        return 0, 1, None, (0, 0, 0, 1), None
    H = x.shape[2]
    if not 0 < x.numel() <= _INT:
        _fits("kda_qk_norm_rope", *x.shape)
    px, sx = _strided(name, x, (B, T, H, D), dt, dev)
    if weight is None:
        return H, 1, px, sx, None
    Hw = weight.shape[0]
    if Hw != 1 and Hw != H:
        raise ValueError("%s_weight has %d rows for %d heads" % (name, Hw, H))
    return H, Hw, px, sx, _ptr(name + "_weight", weight, (Hw, D), _F32, dev)


def _rope(freqs, positions, B, T, dev):
    pp = None if positions is None else _ptr("positions", positions, (B, T), _I32, dev)
    if freqs is None:
        return 0, None, pp
    n = freqs.shape[0]
    if n > 128:
        _fits("kda_qk_norm_rope", 2 * n)
    return 2 * n, _ptr("freqs", freqs, (n,), _F64, dev), pp


def qk_norm_rope_fwd(q, k, freqs, positions=None, norm="rms", q_weight=None, k_weight=None, eps=1e-6, interleaved=False,
                     rope_scale=1.0, q_out=None, k_out=None):
    """Norm over each head's channels (norm "rms", "l2" or None), times q_weight / k_weight (1,D) or (H,D) float32, then
    the rotation by positions (B,T) int32 (None: a token's index) at freqs (R/2,) float64 (rope_frequencies; None: no
    rotation) of the first R channels.  q (B,T,Hq,D) and k (B,T,Hk,D) are views of a projection with any strides but
    the last; k may be None.  Returns (q_out, k_out), (B,Hq,T,D) and (B,Hk,T,D) contiguous."""
    B, T, _, D = q.shape
    dt, dev = q.dtype, q.get_device()
    code, kind = _code(dt), _one_of("norm", norm, _NORMS)
    Hq, Hqw, pq, sq, pqw = _side("q", q, B, T, D, q_weight, dt, dev)
    Hk, Hkw, pk, sk, pkw = _side("k", k, B, T, D, k_weight, dt, dev)
    R, pf, pp = _rope(freqs, positions, B, T, dev)
    po = None if q_out is None else _ptr("q_out", q_out, (B, Hq, T, D), dt, dev)
    pe = None if k is None or k_out is None else _ptr("k_out", k_out, (B, Hk, T, D), dt, dev)
    if dev < 0:
        _gpu(dev)
    if q_out is None:
        q_out = q.new_empty((B, Hq, T, D))
        po = q_out.data_ptr()
    if k is None:
        k_out = None
    elif k_out is None:
        k_out = q.new_empty((B, Hk, T, D))
        pe = k_out.data_ptr()
    _run(dev, "kda_qk_norm_rope_fwd", pq, sq[0], sq[1], sq[2], pk, sk[0], sk[1], sk[2], pqw, Hqw, pkw, Hkw, kind, float(eps), pf, pp,
         float(rope_scale), 1 if interleaved else 0, po, pe, B, T, Hq, Hk, D, R, code)
    return q_out, k_out


def qk_norm_rope_bwd_workspace_bytes(B, T, Hq, Hk, D, q_weight_rows=1, k_weight_rows=1) -> int:
    return _need("kda_qk_norm_rope_bwd_workspace_bytes", B, T, Hq, q_weight_rows, Hk, k_weight_rows, D)


def qk_norm_rope_bwd(q, k, freqs, d_q, d_k, positions=None, norm="rms", q_weight=None, k_weight=None, eps=1e-6,
                     interleaved=False, rope_scale=1.0, dq_out=None, dk_out=None, workspace=None):
    """Adjoint of qk_norm_rope_fwd for cotangents d_q (B,Hq,T,D) and d_k (B,Hk,T,D): dict(dq, dk, dq_weight, dk_weight),
    dq (B,T,Hq,D) and dk (B,T,Hk,D) in d_q's dtype (into dq_out and dk_out, which may be slices of a fused projection's
    gradient), the weights' gradients float32 in the weights' shapes, None without weights.  k and d_k may be None."""
    B, T, _, D = q.shape
    dt, dev = q.dtype, q.get_device()
    code, kind = _code(dt), _one_of("norm", norm, _NORMS)
    Hq, Hqw, pq, sq, pqw = _side("q", q, B, T, D, q_weight, dt, dev)
    Hk, Hkw, pk, sk, pkw = _side("k", k, B, T, D, k_weight, dt, dev)
    R, pf, pp = _rope(freqs, positions, B, T, dev)
    pdq = _ptr("d_q", d_q, (B, Hq, T, D), dt, dev)
    pdk = None if k is None else _ptr("d_k", d_k, (B, Hk, T, D), dt, dev)
    if dq_out is None:
        dq_out = q.new_empty((B, T, Hq, D))
    poq, soq = _strided("dq_out", dq_out, (B, T, Hq, D), dt, dev)
    pok, sok = None, (0, 0, 0, 1)
    if k is None:
        dk_out = None
    else:
        if dk_out is None:
            dk_out = q.new_empty((B, T, Hk, D))
        pok, sok = _strided("dk_out", dk_out, (B, T, Hk, D), dt, dev)
    _gpu(dev)
    dqw = dkw = pgq = pgk = None
    if q_weight is not None:
        dqw = torch.empty_like(q_weight)
        pgq = dqw.data_ptr()
    if k_weight is not None:
        dkw = torch.empty_like(k_weight)
        pgk = dkw.data_ptr()
    need = 0
    if pgq is not None or pgk is not None:
        need = _bytes("kda_qk_norm_rope_bwd_workspace_bytes", B, T, Hq, Hqw, Hk, Hkw, D)
    ws, pws, nws = _workspace(workspace, need, q)
    _run(dev, "kda_qk_norm_rope_bwd", pq, *sq[:3], pk, *sk[:3], pqw, Hqw, pkw, Hkw, kind, float(eps), pf, pp, float(rope_scale),
         int(bool(interleaved)), pdq, pdk, poq, *soq[:3], pok, *sok[:3], pgq, pgk, pws, nws, B, T, Hq, Hk, D, R, code)
    return dict(dq=dq_out, dk=dk_out, dq_weight=dqw, dk_weight=dkw)


def gated_scan_workspace_bytes(B, H, T, D, dtype=torch.bfloat16) -> int:
    return _need("kda_gated_scan_workspace_bytes", B, H, T, D, _code(dtype))


def gated_scan_fwd(x, z, A_log, dt_bias=None, state_in=None, input_gate=None, lengths=None, normalize=True,
                   output_state=True, want_ckpt=False, out=None, state_out=None, workspace=None):
    """Gated linear recurrence h_t = a_t h_{t-1} + n_t sigmoid(input_gate_t) x_t per channel with the decay gate
    a = exp(-exp(A_log) softplus(z + dt_bias)) and n = sqrt(1 - a^2) (1 without normalize): x, z, input_gate (None: no
    gate) (B,H,T,D), A_log (H,), dt_bias (H,D), states (B,H,D) float32.  Returns (y, state_out, ckpt): y_t = h_t,
    state_out None when output_state is False, ckpt (B,H,ceil(T/GATED_SCAN_CHUNK),D) float32 for gated_scan_bwd, None
    without want_ckpt.  lengths (B,) int32 ends each sequence early: y's rows behind it are left as they are in `out`
    (uninitialised without one).  workspace: None allocates what gated_scan_workspace_bytes() asks for."""
    B, H, T, D = x.shape
    dt, dev = x.dtype, x.get_device()
    code = _code(dt)
    if not 0 < x.numel() <= _INT:
        _fits("kda_gated_scan_fwd", B, H, T, D)
    shape, state = (B, H, T, D), (B, H, D)
    px, pz = _ptr("x", x, shape, dt, dev), _ptr("z", z, shape, dt, dev)
    pi = _opt("input_gate", input_gate, shape, dt, dev)
    pa, pb = _ptr("A_log", A_log, (H,), _F32, dev), _opt("dt_bias", dt_bias, (H, D), _F32, dev)
    ps, pn = _opt("state_in", state_in, state, _F32, dev), _opt("lengths", lengths, (B,), _I32, dev)
    po, pe = _opt("out", out, shape, dt, dev), _opt("state_out", state_out, state, _F32, dev)
    _gpu(dev)
    if out is None:
        out = torch.empty_like(x)
        po = out.data_ptr()
    if not output_state:
        state_out = pe = None
    elif state_out is None:
        state_out = A_log.new_empty(state)
        pe = state_out.data_ptr()
    ckpt = pc = None
    if want_ckpt:
        ckpt = A_log.new_empty((B, H, -(-T // GATED_SCAN_CHUNK), D))
        pc = ckpt.data_ptr()
    ws, pw, nw = _workspace(workspace, _bytes("kda_gated_scan_workspace_bytes", B, H, T, D, code), A_log)
    _run(dev, "kda_gated_scan_fwd", px, pz, pa, pb, pi, pn, ps, int(bool(normalize)), po, pe, pc, pw, nw, B, H, T, D, code)
    return out, state_out, ckpt


def gated_scan_step(x, z, A_log, dt_bias, state, input_gate=None, normalize=True, out=None):
    """One token per channel: x, z, input_gate (B,H,D).  Updates `state` (B,H,D) float32 in place and returns y (B,H,D)."""
    shape, dt, dev = x.shape, x.dtype, x.get_device()
    B, H, D = shape
    code = _code(dt)
    if not 0 < x.numel() <= _INT:
        _fits("kda_gated_scan_step", B, H, D)
    pi = None if input_gate is None else _ptr("input_gate", input_gate, shape, dt, dev)
    pb = None if dt_bias is None else _ptr("dt_bias", dt_bias, (H, D), _F32, dev)
    px, pz, pa = _ptr("x", x, shape, dt, dev), _ptr("z", z, shape, dt, dev), _ptr("A_log", A_log, (H,), _F32, dev)
    ps = _ptr("state", state, shape, _F32, dev)
    po = None if out is None else _ptr("out", out, shape, dt, dev)
    if dev < 0:
        _gpu(dev)
    if po is None:
        out = torch.empty_like(x)
        po = out.data_ptr()
    _run(dev, "kda_gated_scan_step", px, pz, pa, pb, pi, 1 if normalize else 0, ps, po, B, H, D, code)
    return out


def gated_scan_bwd_workspace_bytes(B, H, T, D, dtype=torch.bfloat16) -> int:
    return _need("kda_gated_scan_bwd_workspace_bytes", B, H, T, D, _code(dtype))


def gated_scan_bwd(x, z, A_log, dt_bias, ckpt, dy, d_state_out=None, input_gate=None, lengths=None, normalize=True,
                   workspace=None):
    """Gradients of sum(y * dy) + sum(state_out * d_state_out) from gated_scan_fwd's inputs and its ckpt:
    dict(dx, dz, dinput_gate, dA_log, ddt_bias, dstate_in), the first three in dy's dtype (dinput_gate None without an
    input gate), the rest float32.  Rows behind a sequence's length get zero gradients."""
    B, H, T, D = x.shape
    dt, dev = x.dtype, x.get_device()
    code = _code(dt)
    if not 0 < x.numel() <= _INT:
        _fits("kda_gated_scan_bwd", B, H, T, D)
    shape, state = (B, H, T, D), (B, H, D)
    px, pz, pd = _ptr("x", x, shape, dt, dev), _ptr("z", z, shape, dt, dev), _ptr("dy", dy, shape, dt, dev)
    pi = _opt("input_gate", input_gate, shape, dt, dev)
    pa, pb = _ptr("A_log", A_log, (H,), _F32, dev), _opt("dt_bias", dt_bias, (H, D), _F32, dev)
    pc = _ptr("ckpt", ckpt, (B, H, -(-T // GATED_SCAN_CHUNK), D), _F32, dev)
    pe, pn = _opt("d_state_out", d_state_out, state, _F32, dev), _opt("lengths", lengths, (B,), _I32, dev)
    _gpu(dev)
    dx, dz = torch.empty_like(x), torch.empty_like(x)
    di = pdi = None
    if input_gate is not None:
        di = torch.empty_like(x)
        pdi = di.data_ptr()
    dA, db, ds = torch.empty_like(A_log), A_log.new_empty((H, D)), A_log.new_empty(state)
    ws, pw, nw = _workspace(workspace, _bytes("kda_gated_scan_bwd_workspace_bytes", B, H, T, D, code), A_log)
    _run(dev, "kda_gated_scan_bwd", px, pz, pa, pb, pi, pn, int(bool(normalize)), pc, pd, pe, dx.data_ptr(), dz.data_ptr(),
         pdi, dA.data_ptr(), db.data_ptr(), ds.data_ptr(), pw, nw, B, H, T, D, code)
    return dict(dx=dx, dz=dz, dinput_gate=di, dA_log=dA, ddt_bias=db, dstate_in=ds)
