"""Operators of a linear-attention layer beside the delta rule: attention with a constant decay per
head (prompts, single tokens, gradients), the layer norm of its read with its backward, and the 8-bit
form in which a training step keeps activations for the backward pass.

Argument marshalling only, as in the package's root: the arithmetic is in the library's HIP kernels.
Layouts are head-major and contiguous.  Every tensor of a call lives on one GPU; the call runs on that
GPU's current stream whatever the current device is.
"""
from __future__ import annotations

import torch

from . import _call, _check_f32, _check_out, _dtype_code, _lib, _ptr, _stream, read_scale

__all__ = ["decay_attn_workspace_bytes", "decay_attn_fwd", "decay_attn_step", "decay_attn_bwd_workspace_bytes",
           "decay_attn_bwd", "layer_norm_fwd", "layer_norm_bwd_workspace_bytes", "layer_norm_bwd", "ckpt_pack",
           "ckpt_unpack"]


def _code(dtype):
    if dtype == torch.bfloat16:
        return _lib.KDA_BF16
    if dtype == torch.float32:
        return _lib.KDA_F32
    raise TypeError("activations must be float32 or bfloat16, got %s" % dtype)


def _same_device(dev, **tensors):
    for name, t in tensors.items():
        if t is not None and t.device != dev:
            raise ValueError("%s is on %s, expected %s" % (name, t.device, dev))


def _run(dev, fn, *args):
    """The call on dev's current stream, with dev current while it launches."""
    if dev.index is None or dev.index == torch.cuda.current_device():
        return _call(fn, *args, _stream(dev))
    with torch.cuda.device(dev):
        return _call(fn, *args, _stream(dev))


def _act(name, t, shape, dtype):
    if tuple(t.shape) != tuple(shape):
        raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), tuple(shape)))
    if t.dtype != dtype:
        raise TypeError("%s has dtype %s, expected %s" % (name, t.dtype, dtype))


def _workspace(workspace, need, dev):
    """(tensor or None, its bytes): the caller's, or `need` bytes from torch's caching allocator."""
    if workspace is None:
        if not need:
            return None, 0
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    _same_device(dev, workspace=workspace)
    return workspace, workspace.numel() * workspace.element_size()


def _lengths(lengths, B):
    if lengths is None:
        return
    if lengths.dtype != torch.int32:
        raise TypeError("lengths must be int32")
    if tuple(lengths.shape) != (B,):
        raise ValueError("lengths has shape %s, expected %s" % (tuple(lengths.shape), (B,)))


def decay_attn_workspace_bytes(B, H, T, K, V, dtype=torch.bfloat16) -> int:
    return int(_lib.load().kda_decay_attn_workspace_bytes(B, H, T, K, V, _code(dtype)))


def decay_attn_fwd(q, k, v, log_decay, state_in=None, lengths=None, scale=None, output_state=True, out=None,
                   state_out=None, workspace=None):
    """Linear attention S_t = exp(log_decay[h]) S_{t-1} + k_t v_t^T, o_t = scale S_t^T q_t over prompts:
    q, k (B,H,T,K), v (B,H,T,V), log_decay (H,) float32 <= 0.  Returns (o, state_out); state_out is None
    when output_state is False.  lengths (B,) int32 ends each sequence early: o's rows behind it are left
    as they are in `out` (uninitialised without one).  scale=None means K**-0.5.  workspace: None
    allocates what decay_attn_workspace_bytes() asks for, or a uint8 tensor of at least that size."""
    B, H, T, K = q.shape
    V = v.shape[-1]
    _act("k", k, (B, H, T, K), q.dtype)
    _act("v", v, (B, H, T, V), q.dtype)
    _check_f32("log_decay", log_decay, (H,))
    _check_f32("state_in", state_in, (B, H, K, V))
    _lengths(lengths, B)
    dev = q.device
    _same_device(dev, k=k, v=v, log_decay=log_decay, state_in=state_in, lengths=lengths)
    code = _dtype_code(q)
    _check_out("out", out, (B, H, T, V), q.dtype, dev)
    _check_out("state_out", state_out, (B, H, K, V), torch.float32, dev)
    o = out if out is not None else torch.empty((B, H, T, V), dtype=q.dtype, device=dev)
    if not output_state:
        state_out = None
    elif state_out is None:
        state_out = torch.empty((B, H, K, V), dtype=torch.float32, device=dev)
    ws, nws = _workspace(workspace, int(_lib.load().kda_decay_attn_workspace_bytes(B, H, T, K, V, code)), dev)
    _run(dev, "kda_decay_attn_fwd", _ptr(q), _ptr(k), _ptr(v), _ptr(log_decay), _ptr(lengths), _ptr(state_in),
         read_scale(K) if scale is None else float(scale), _ptr(o), _ptr(state_out), _ptr(ws), nws, B, H, T, K, V,
         code)
    return o, state_out


def decay_attn_step(q, k, v, log_decay, state, scale=None, out=None):
    """One token per head: q, k (B,H,K), v (B,H,V).  Updates `state` (B,H,K,V) float32 in place and
    returns o (B,H,V)."""
    B, H, K = q.shape
    V = v.shape[-1]
    _act("k", k, (B, H, K), q.dtype)
    _act("v", v, (B, H, V), q.dtype)
    _check_f32("log_decay", log_decay, (H,))
    if state is None:
        raise TypeError("state must be a torch.Tensor")
    _check_f32("state", state, (B, H, K, V))
    dev = q.device
    _same_device(dev, k=k, v=v, log_decay=log_decay, state=state)
    _check_out("out", out, (B, H, V), q.dtype, dev)
    o = out if out is not None else torch.empty((B, H, V), dtype=q.dtype, device=dev)
    _run(dev, "kda_decay_attn_step", _ptr(q), _ptr(k), _ptr(v), _ptr(log_decay), _ptr(state),
         read_scale(K) if scale is None else float(scale), _ptr(o), B, H, K, V, _dtype_code(q))
    return o


def decay_attn_bwd_workspace_bytes(B, H, T, K, V, dtype=torch.bfloat16) -> int:
    return int(_lib.load().kda_decay_attn_bwd_workspace_bytes(B, H, T, K, V, _code(dtype)))


def _kept(name, x, shape, dtype):
    """(tensor, scales or None) of an activation, or of its 8-bit form (codes, scales)."""
    if not isinstance(x, (tuple, list)):
        _act(name, x, shape, dtype)
        return x, None
    codes, scales = x
    _act(name + " codes", codes, shape, torch.uint8)
    D = shape[-1]
    _act(name + " scales", scales, tuple(shape[:-1]) + (max(1, D // 32),), torch.uint8)
    return codes, scales


def decay_attn_bwd(q, k, v, log_decay, state_in, d_o, d_state_out=None, lengths=None, scale=None, workspace=None):
    """Gradients of sum(o * d_o) + sum(state_out * d_state_out): dict(dq, dk, dv, dstate_in), the first
    three in d_o's dtype, dstate_in float32.  q, k and v are tensors in d_o's dtype or the (codes, scales)
    of ckpt_pack.  Rows behind a sequence's length get zero gradients."""
    qt = q[0] if isinstance(q, (tuple, list)) else q
    B, H, T, K = qt.shape
    V = d_o.shape[-1]
    dt, dev = d_o.dtype, d_o.device
    code = _dtype_code(d_o)
    _act("d_o", d_o, (B, H, T, V), dt)
    (q, qs), (k, ks), (v, vs) = (_kept("q", q, (B, H, T, K), dt), _kept("k", k, (B, H, T, K), dt),
                                 _kept("v", v, (B, H, T, V), dt))
    _check_f32("log_decay", log_decay, (H,))
    _check_f32("state_in", state_in, (B, H, K, V))
    _check_f32("d_state_out", d_state_out, (B, H, K, V))
    _lengths(lengths, B)
    _same_device(dev, q=q, k=k, v=v, q_scales=qs, k_scales=ks, v_scales=vs, log_decay=log_decay, state_in=state_in,
                 d_state_out=d_state_out, lengths=lengths)
    out = dict(dq=torch.empty((B, H, T, K), dtype=dt, device=dev), dk=torch.empty((B, H, T, K), dtype=dt, device=dev),
               dv=torch.empty((B, H, T, V), dtype=dt, device=dev),
               dstate_in=torch.empty((B, H, K, V), dtype=torch.float32, device=dev))
    ws, nws = _workspace(workspace, int(_lib.load().kda_decay_attn_bwd_workspace_bytes(B, H, T, K, V, code)), dev)
    _run(dev, "kda_decay_attn_bwd", _ptr(q), _ptr(k), _ptr(v), _ptr(qs), _ptr(ks), _ptr(vs), _ptr(log_decay),
         _ptr(lengths), _ptr(state_in), read_scale(K) if scale is None else float(scale), _ptr(d_o),
         _ptr(d_state_out), _ptr(out["dq"]), _ptr(out["dk"]), _ptr(out["dv"]), _ptr(out["dstate_in"]), _ptr(ws), nws,
         B, H, T, K, V, code)
    return out


def layer_norm_fwd(x, weight=None, bias=None, eps=1e-5, want_stats=True, out=None):
    """Layer norm over the last axis of x (B,H,T,D) with weight and bias (H,D) float32 (None: ones and
    zeros).  Returns (y, mean, rstd), the statistics (B,H,T) float32 or None without want_stats."""
    B, H, T, D = x.shape
    _check_f32("weight", weight, (H, D))
    _check_f32("bias", bias, (H, D))
    dev = x.device
    _same_device(dev, weight=weight, bias=bias)
    _check_out("out", out, (B, H, T, D), x.dtype, dev)
    code = _dtype_code(x)
    y = out if out is not None else torch.empty_like(x)
    mean = torch.empty((B, H, T), dtype=torch.float32, device=dev) if want_stats else None
    rstd = torch.empty((B, H, T), dtype=torch.float32, device=dev) if want_stats else None
    _run(dev, "kda_layer_norm_fwd", _ptr(x), _ptr(weight), _ptr(bias), float(eps), _ptr(y), _ptr(mean), _ptr(rstd),
         B, H, T, D, code)
    return y, mean, rstd


def layer_norm_bwd_workspace_bytes(B, H, T, D, dtype=torch.bfloat16) -> int:
    return int(_lib.load().kda_layer_norm_bwd_workspace_bytes(B, H, T, D, _code(dtype)))


def layer_norm_bwd(x, weight, mean, rstd, dy, want_params=True, workspace=None, dx_out=None):
    """Adjoint of layer_norm_fwd for a cotangent dy on y, from its mean and rstd: (dx, dweight, dbias), dx
    in dy's dtype, the sums (H,D) float32 (None without want_params).  x is the tensor or the (codes,
    scales) of ckpt_pack; dx_out may be dy itself (computed in place)."""
    B, H, T, D = dy.shape
    dt, dev = dy.dtype, dy.device
    code = _dtype_code(dy)
    x, xs = _kept("x", x, (B, H, T, D), dt)
    _check_f32("weight", weight, (H, D))
    for name, t in (("mean", mean), ("rstd", rstd)):
        if t is None:
            raise TypeError("%s must be a torch.Tensor" % name)
        _check_f32(name, t, (B, H, T))
    _same_device(dev, x=x, x_scales=xs, weight=weight, mean=mean, rstd=rstd)
    _check_out("dx_out", dx_out, (B, H, T, D), dt, dev)
    dx = dx_out if dx_out is not None else torch.empty_like(dy)
    dw = torch.empty((H, D), dtype=torch.float32, device=dev) if want_params else None
    db = torch.empty((H, D), dtype=torch.float32, device=dev) if want_params else None
    need = int(_lib.load().kda_layer_norm_bwd_workspace_bytes(B, H, T, D, code)) if want_params else 0
    ws, nws = _workspace(workspace, need, dev)
    _run(dev, "kda_layer_norm_bwd", _ptr(x), _ptr(xs), _ptr(weight), _ptr(mean), _ptr(rstd), _ptr(dy), _ptr(dx),
         _ptr(dw), _ptr(db), _ptr(ws), nws, B, H, T, D, code)
    return dx, dw, db


def ckpt_pack(x):
    """x (..., D) in 8 bits: (codes uint8 of x's shape, scales uint8 (..., max(1, D // 32))), e4m3 values
    with one power-of-two scale per group of min(D, 32) channels.  D <= 32 or a multiple of 32."""
    D = x.shape[-1]
    code = _dtype_code(x)
    codes = torch.empty(x.shape, dtype=torch.uint8, device=x.device)
    scales = torch.empty(tuple(x.shape[:-1]) + (max(1, D // 32),), dtype=torch.uint8, device=x.device)
    _run(x.device, "kda_ckpt_pack", _ptr(x), _ptr(codes), _ptr(scales), x.numel() // D if D else 0, D, code)
    return codes, scales


def ckpt_unpack(codes, scales, dtype=torch.bfloat16, out=None):
    """The values that ckpt_pack's codes and scales stand for, in dtype."""
    D = codes.shape[-1]
    code = _code(dtype)
    _act("codes", codes, codes.shape, torch.uint8)
    _act("scales", scales, tuple(codes.shape[:-1]) + (max(1, D // 32),), torch.uint8)
    dev = codes.device
    _same_device(dev, scales=scales)
    _check_out("out", out, codes.shape, dtype, dev)
    x = out if out is not None else torch.empty(codes.shape, dtype=dtype, device=dev)
    _run(dev, "kda_ckpt_unpack", _ptr(codes), _ptr(scales), _ptr(x), codes.numel() // D if D else 0, D, code)
    return x
