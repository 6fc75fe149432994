"""Operators of a linear-attention layer beside the delta rule: attention with a constant decay per
head (prompts, single tokens, gradients), the layer norm of its read with its backward, and the 8-bit
form in which a training step keeps activations for the backward pass.

Argument marshalling only, as in the package's root: the arithmetic is in the library's HIP kernels.
Layouts are head-major and contiguous.  Every tensor of a call lives on one GPU; the call runs on that
GPU's current stream whatever the current device is.  A decode step's kernel takes a few microseconds,
so a call checks each tensor in one expression and looks at what is wrong only if something is.
"""
from __future__ import annotations

from functools import lru_cache

import torch

from . import _lib, KdaError

__all__ = ["decay_attn_workspace_bytes", "decay_attn_fwd", "decay_attn_step", "decay_attn_bwd_workspace_bytes",
           "decay_attn_bwd", "layer_norm_fwd", "layer_norm_bwd_workspace_bytes", "layer_norm_bwd", "ckpt_pack",
           "ckpt_unpack"]

_F32, _U8, _I32 = torch.float32, torch.uint8, torch.int32
_CODES = {torch.float32: _lib.KDA_F32, torch.bfloat16: _lib.KDA_BF16}


def _code(dtype):
    code = _CODES.get(dtype)
    if code is None:
        raise TypeError("activations must be float32 or bfloat16, got %s" % dtype)
    return code


def _refuse(name, t, shape, dtype, dev):
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if tuple(t.shape) != tuple(shape):
        raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), tuple(shape)))
    if t.dtype != dtype:
        raise TypeError("%s has dtype %s, expected %s" % (name, t.dtype, dtype))
    if t.get_device() != dev:
        raise ValueError("%s is on %s, the call's tensors on GPU %d" % (name, t.device, dev))
    raise ValueError("%s must be contiguous" % name)


def _ptr(name, t, shape, dtype, dev):
    """Address of a tensor that must have exactly this shape, dtype and device."""
    try:
        if t.shape == shape and t.dtype is dtype and t.get_device() == dev and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    _refuse(name, t, shape, dtype, dev)


def _opt(name, t, shape, dtype, dev):
    return None if t is None else _ptr(name, t, shape, dtype, dev)


def _run(dev, fn, *args):
    """The call on GPU dev's current stream, with dev current while it launches."""
    fn_ = getattr(_lib.load(), fn)
    if dev == torch.cuda.current_device():
        st = fn_(*args, torch._C._cuda_getCurrentRawStream(dev))
    else:
        with torch.cuda.device(dev):
            st = fn_(*args, torch._C._cuda_getCurrentRawStream(dev))
    if st != _lib.KDA_OK:
        raise KdaError(fn, st)


def _gpu(dev):
    if dev < 0:
        raise ValueError("tensors must live on the GPU")


@lru_cache(maxsize=None)
def _scale_of(K):
    return float(_lib.load().kda_read_scale(K))


@lru_cache(maxsize=4096)
def _bytes(fn, *sizes):
    return int(getattr(_lib.load(), fn)(*sizes))


def _workspace(workspace, need, dev):
    """(tensor kept alive, address, bytes): the caller's, or `need` bytes from torch's caching allocator."""
    if workspace is None:
        if not need:
            return None, None, 0
        workspace = torch.empty(need, dtype=_U8, device=dev)
    elif workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous and on the call's GPU")
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


def decay_attn_workspace_bytes(B, H, T, K, V, dtype=torch.bfloat16) -> int:
    return _bytes("kda_decay_attn_workspace_bytes", B, H, T, K, V, _code(dtype))


def decay_attn_fwd(q, k, v, log_decay, state_in=None, lengths=None, scale=None, output_state=True, out=None,
                   state_out=None, workspace=None):
    """Linear attention S_t = exp(log_decay[h]) S_{t-1} + k_t v_t^T, o_t = scale S_t^T q_t over prompts:
    q, k (B,H,T,K), v (B,H,T,V), log_decay (H,) float32 <= 0.  Returns (o, state_out); state_out is None
    when output_state is False.  lengths (B,) int32 ends each sequence early: o's rows behind it are left
    as they are in `out` (uninitialised without one).  scale=None means K**-0.5.  workspace: None
    allocates what decay_attn_workspace_bytes() asks for, or a uint8 tensor of at least that size."""
    B, H, T, K = q.shape
    V = v.shape[-1]
    dt, dev = q.dtype, q.get_device()
    code = _code(dt)
    shape, state = (B, H, T, V), (B, H, K, V)
    pq, pk, pv = _ptr("q", q, (B, H, T, K), dt, dev), _ptr("k", k, (B, H, T, K), dt, dev), _ptr("v", v, shape, dt, dev)
    pg = _ptr("log_decay", log_decay, (H,), _F32, dev)
    ps = _opt("state_in", state_in, state, _F32, dev)
    pn = _opt("lengths", lengths, (B,), _I32, dev)
    po = _opt("out", out, shape, dt, dev)
    pe = _opt("state_out", state_out, state, _F32, dev)
    _gpu(dev)
    if out is None:
        out = torch.empty_like(v)
        po = out.data_ptr()
    if not output_state:
        state_out = pe = None
    elif state_out is None:
        state_out = torch.empty(state, dtype=_F32, device=dev)
        pe = state_out.data_ptr()
    ws, pw, nw = _workspace(workspace, _bytes("kda_decay_attn_workspace_bytes", B, H, T, K, V, code), dev)
    _run(dev, "kda_decay_attn_fwd", pq, pk, pv, pg, pn, ps, _scale_of(K) if scale is None else float(scale), po, pe,
         pw, nw, B, H, T, K, V, code)
    return out, state_out


def decay_attn_step(q, k, v, log_decay, state, scale=None, out=None):
    """One token per head: q, k (B,H,K), v (B,H,V).  Updates `state` (B,H,K,V) float32 in place and
    returns o (B,H,V)."""
    B, H, K = q.shape
    V = v.shape[-1]
    dt, dev = q.dtype, q.get_device()
    code = _code(dt)
    shape = (B, H, V)
    pq, pk, pv = _ptr("q", q, (B, H, K), dt, dev), _ptr("k", k, (B, H, K), dt, dev), _ptr("v", v, shape, dt, dev)
    pg = _ptr("log_decay", log_decay, (H,), _F32, dev)
    ps = _ptr("state", state, (B, H, K, V), _F32, dev)
    po = _opt("out", out, shape, dt, dev)
    _gpu(dev)
    if out is None:
        out = torch.empty_like(v)
        po = out.data_ptr()
    _run(dev, "kda_decay_attn_step", pq, pk, pv, pg, ps, _scale_of(K) if scale is None else float(scale), po, B, H, K,
         V, code)
    return out


def decay_attn_bwd_workspace_bytes(B, H, T, K, V, dtype=torch.bfloat16) -> int:
    return _bytes("kda_decay_attn_bwd_workspace_bytes", B, H, T, K, V, _code(dtype))


def _kept(name, x, shape, dtype, dev):
    """Addresses (tensor, scales or None) of an activation, or of its 8-bit form (codes, scales)."""
    if not isinstance(x, (tuple, list)):
        return _ptr(name, x, shape, dtype, dev), None
    codes, scales = x
    return (_ptr(name + " codes", codes, shape, _U8, dev),
            _ptr(name + " scales", scales, shape[:-1] + (max(1, shape[-1] // 32),), _U8, dev))


def decay_attn_bwd(q, k, v, log_decay, state_in, d_o, d_state_out=None, lengths=None, scale=None, workspace=None):
    """Gradients of sum(o * d_o) + sum(state_out * d_state_out): dict(dq, dk, dv, dstate_in), the first
    three in d_o's dtype, dstate_in float32.  q, k and v are tensors in d_o's dtype, or all three the
    (codes, scales) of ckpt_pack.  Rows behind a sequence's length get zero gradients."""
    B, H, T, K = (q[0] if isinstance(q, (tuple, list)) else q).shape
    V = d_o.shape[-1]
    dt, dev = d_o.dtype, d_o.get_device()
    code = _code(dt)
    kshape, vshape, state = (B, H, T, K), (B, H, T, V), (B, H, K, V)
    pd = _ptr("d_o", d_o, vshape, dt, dev)
    (pq, sq), (pk, sk), (pv, sv) = (_kept("q", q, kshape, dt, dev), _kept("k", k, kshape, dt, dev),
                                    _kept("v", v, vshape, dt, dev))
    if (sq is None) != (sk is None) or (sq is None) != (sv is None):
        raise TypeError("q, k and v are tensors, or all three (codes, scales)")
    pg = _ptr("log_decay", log_decay, (H,), _F32, dev)
    ps = _opt("state_in", state_in, state, _F32, dev)
    pe = _opt("d_state_out", d_state_out, state, _F32, dev)
    pn = _opt("lengths", lengths, (B,), _I32, dev)
    _gpu(dev)
    dq, dk = torch.empty(kshape, dtype=dt, device=dev), torch.empty(kshape, dtype=dt, device=dev)
    dv, ds = torch.empty(vshape, dtype=dt, device=dev), torch.empty(state, dtype=_F32, device=dev)
    ws, pw, nw = _workspace(workspace, _bytes("kda_decay_attn_bwd_workspace_bytes", B, H, T, K, V, code), dev)
    _run(dev, "kda_decay_attn_bwd", pq, pk, pv, sq, sk, sv, pg, pn, ps, _scale_of(K) if scale is None else float(scale),
         pd, pe, dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), ds.data_ptr(), pw, nw, B, H, T, K, V, code)
    return dict(dq=dq, dk=dk, dv=dv, dstate_in=ds)


def layer_norm_fwd(x, weight=None, bias=None, eps=1e-5, want_stats=True, out=None):
    """Layer norm over the last axis of x (B,H,T,D) with weight and bias (H,D) float32 (None: ones and
    zeros).  Returns (y, mean, rstd), the statistics (B,H,T) float32 or None without want_stats."""
    B, H, T, D = x.shape
    dt, dev = x.dtype, x.get_device()
    code = _code(dt)
    shape = (B, H, T, D)
    px = _ptr("x", x, shape, dt, dev)
    pw, pb = _opt("weight", weight, (H, D), _F32, dev), _opt("bias", bias, (H, D), _F32, dev)
    py = _opt("out", out, shape, dt, dev)
    _gpu(dev)
    if out is None:
        out = torch.empty_like(x)
        py = out.data_ptr()
    mean = rstd = pm = pr = None
    if want_stats:
        mean, rstd = torch.empty((2, B, H, T), dtype=_F32, device=dev).unbind(0)
        pm, pr = mean.data_ptr(), rstd.data_ptr()
    _run(dev, "kda_layer_norm_fwd", px, pw, pb, float(eps), py, pm, pr, B, H, T, D, code)
    return out, mean, rstd


def layer_norm_bwd_workspace_bytes(B, H, T, D, dtype=torch.bfloat16) -> int:
    return _bytes("kda_layer_norm_bwd_workspace_bytes", B, H, T, D, _code(dtype))


def layer_norm_bwd(x, weight, mean, rstd, dy, want_params=True, workspace=None, dx_out=None):
    """Adjoint of layer_norm_fwd for a cotangent dy on y, from its mean and rstd: (dx, dweight, dbias), dx
    in dy's dtype, the sums (H,D) float32 (None without want_params).  x is the tensor or the (codes,
    scales) of ckpt_pack; dx_out may be dy itself (computed in place)."""
    B, H, T, D = dy.shape
    dt, dev = dy.dtype, dy.get_device()
    code = _code(dt)
    shape, rows = (B, H, T, D), (B, H, T)
    pd = _ptr("dy", dy, shape, dt, dev)
    px, sx = _kept("x", x, shape, dt, dev)
    pw = _opt("weight", weight, (H, D), _F32, dev)
    pm, pr = _ptr("mean", mean, rows, _F32, dev), _ptr("rstd", rstd, rows, _F32, dev)
    pdx = _opt("dx_out", dx_out, shape, dt, dev)
    _gpu(dev)
    if dx_out is None:
        dx_out = torch.empty_like(dy)
        pdx = dx_out.data_ptr()
    dw = db = pdw = pdb = None
    need = 0
    if want_params:
        dw, db = torch.empty((2, H, D), dtype=_F32, device=dev).unbind(0)
        pdw, pdb = dw.data_ptr(), db.data_ptr()
        need = _bytes("kda_layer_norm_bwd_workspace_bytes", B, H, T, D, code)
    ws, pws, nws = _workspace(workspace, need, dev)
    _run(dev, "kda_layer_norm_bwd", px, sx, pw, pm, pr, pd, pdx, pdw, pdb, pws, nws, B, H, T, D, code)
    return dx_out, dw, db


def ckpt_pack(x):
    """x (..., D) in 8 bits: (codes uint8 of x's shape, scales uint8 (..., max(1, D // 32))), e4m3 values
    with one power-of-two scale per group of min(D, 32) channels.  D <= 32 or a multiple of 32."""
    shape, dev = tuple(x.shape), x.get_device()
    D = shape[-1]
    code = _code(x.dtype)
    px = _ptr("x", x, shape, x.dtype, dev)
    _gpu(dev)
    codes = torch.empty(shape, dtype=_U8, device=dev)
    scales = torch.empty(shape[:-1] + (max(1, D // 32),), dtype=_U8, device=dev)
    _run(dev, "kda_ckpt_pack", px, codes.data_ptr(), scales.data_ptr(), x.numel() // max(D, 1), D, code)
    return codes, scales


def ckpt_unpack(codes, scales, dtype=torch.bfloat16, out=None):
    """The values that ckpt_pack's codes and scales stand for, in dtype."""
    shape, dev = tuple(codes.shape), codes.get_device()
    D = shape[-1]
    code = _code(dtype)
    pc = _ptr("codes", codes, shape, _U8, dev)
    ps = _ptr("scales", scales, shape[:-1] + (max(1, D // 32),), _U8, dev)
    px = _opt("out", out, shape, dtype, dev)
    _gpu(dev)
    if out is None:
        out = torch.empty(shape, dtype=dtype, device=dev)
        px = out.data_ptr()
    _run(dev, "kda_ckpt_unpack", pc, ps, px, codes.numel() // max(D, 1), D, code)
    return out
