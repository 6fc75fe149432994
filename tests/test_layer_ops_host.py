"""Refusals of the decay attention, the layer norm and the 8-bit activations: every argument error is
reported before anything is launched.  The calls pass fake device addresses, so they run only where no
GPU is visible."""
import ctypes

import pytest
import torch

import gated_delta_rule_47_amd as kda
from gated_delta_rule_47_amd import _lib


def _gpu_visible():
    try:
        return torch.cuda.is_available()
    except Exception:
        return False


cpu_only = pytest.mark.skipif(_gpu_visible(), reason="fake device pointers: CPU-only check")
P = ctypes.c_void_p
NULL, SHAPE, DTYPE, ALIAS, WORKSPACE, ALIGN = -1, -2, -3, -5, -7, -8
F32, BF16 = 0, 1


def _at(i):
    return P(0x10000000 * (i + 1))


def _rejected():
    return kda.counters()["rejected"]


def test_workspace_bytes():
    lib = _lib.load()
    f, b = lib.kda_decay_attn_workspace_bytes, lib.kda_decay_attn_bwd_workspace_bytes
    assert f(4, 32, 16384, 128, 128, BF16) == 0                  # heads x value tiles fill the chip
    one = f(1, 4, 30011, 128, 128, BF16)
    assert one > 0 and one % (4 * 128 * 128 * 4) == 0 and b(1, 4, 30011, 128, 128, BF16) == 2 * one
    assert f(1, 1, 64, 64, 64, BF16) == 0 and f(1, 1, 0, 64, 64, BF16) == 0
    for args in ((0, 1, 4096, 64, 64, BF16), (1, 1, -1, 64, 64, BF16), (1, 1, 4096, 48, 64, BF16),
                 (1, 1, 4096, 64, 64, 7), (1, 1, 1 << 24, 128, 128, BF16)):
        assert f(*args) == 0 and b(*args) == 0
    n = lib.kda_layer_norm_bwd_workspace_bytes
    assert n(1, 1, 32768, 512, BF16) % (2 * 512 * 4) == 0 and n(1, 1, 32768, 512, BF16) > 0
    assert n(1, 1, 0, 512, BF16) == 0 and n(1, 1, 5, 0, BF16) == 0 and n(1, 1, 5, 8, 3) == 0


@cpu_only
def test_decay_attn_fwd_refusals():
    f = _lib.load().kda_decay_attn_fwd
    q, k, v, g, n, s0, o, s1, ws = (_at(i) for i in range(9))
    ok = dict(q=q, k=k, v=v, g=g, n=n, s0=s0, scale=1.0, o=o, s1=s1, ws=ws, nws=1 << 26, B=1, H=4, T=4096, K=128,
              V=128, dt=BF16)

    def call(**kw):
        a = {**ok, **kw}
        return f(a["q"], a["k"], a["v"], a["g"], a["n"], a["s0"], a["scale"], a["o"], a["s1"], a["ws"], a["nws"],
                 a["B"], a["H"], a["T"], a["K"], a["V"], a["dt"], None)

    cases = [(dict(q=None), NULL), (dict(k=None), NULL), (dict(v=None), NULL), (dict(g=None), NULL),
             (dict(o=None), NULL), (dict(dt=5), DTYPE), (dict(B=0), SHAPE), (dict(H=0), SHAPE), (dict(T=-1), SHAPE),
             (dict(K=12), SHAPE), (dict(V=256), SHAPE), (dict(T=1 << 23), SHAPE), (dict(B=1 << 13, H=1 << 13), SHAPE),
             (dict(B=1 << 11, H=1 << 10, T=1), SHAPE),
             (dict(q=P(q.value + 8)), ALIGN), (dict(o=P(o.value + 2)), ALIGN), (dict(ws=None), WORKSPACE),
             (dict(nws=1000), WORKSPACE), (dict(ws=P(ws.value + 16)), ALIGN), (dict(o=q), ALIAS),
             (dict(o=P(v.value + 16)), ALIAS), (dict(s1=k), ALIAS), (dict(s1=o), ALIAS), (dict(s1=g), ALIAS),
             (dict(s1=P(s0.value + 256)), ALIAS), (dict(o=s0), ALIAS), (dict(ws=o), ALIAS), (dict(ws=s0), ALIAS),
             (dict(o=n), ALIAS)]
    before = _rejected()
    for kw, status in cases:
        assert call(**kw) == status, kw
    assert _rejected() - before == len(cases)


@cpu_only
def test_decay_attn_step_refusals():
    f = _lib.load().kda_decay_attn_step
    q, k, v, g, s, o = (_at(i) for i in range(6))
    ok = dict(q=q, k=k, v=v, g=g, s=s, o=o, B=1, H=2, K=16, V=16, dt=F32)

    def call(**kw):
        a = {**ok, **kw}
        return f(a["q"], a["k"], a["v"], a["g"], a["s"], 1.0, a["o"], a["B"], a["H"], a["K"], a["V"], a["dt"], None)

    for name in ("q", "k", "v", "g", "s", "o"):
        assert call(**{name: None}) == NULL, name
    for kw, status in ((dict(dt=2), DTYPE), (dict(K=24), SHAPE), (dict(B=0), SHAPE), (dict(o=q), ALIAS),
                       (dict(o=s), ALIAS), (dict(s=k), ALIAS), (dict(s=g), ALIAS), (dict(s=P(s.value + 4)), ALIGN),
                       (dict(v=P(v.value + 8)), ALIGN), (dict(o=P(o.value + 1)), ALIGN)):
        assert call(**kw) == status, kw


@cpu_only
def test_decay_attn_bwd_refusals():
    f = _lib.load().kda_decay_attn_bwd
    q, k, v, qs, ks, vs, g, n, s0, do, ds, dq, dk, dv, d0, ws = (_at(i) for i in range(16))
    ok = dict(q=q, k=k, v=v, qs=None, ks=None, vs=None, g=g, n=n, s0=s0, do=do, ds=ds, dq=dq, dk=dk, dv=dv, d0=d0,
              ws=ws, nws=1 << 27, B=1, H=2, T=4096, K=64, V=64, dt=BF16)

    def call(**kw):
        a = {**ok, **kw}
        return f(a["q"], a["k"], a["v"], a["qs"], a["ks"], a["vs"], a["g"], a["n"], a["s0"], 1.0, a["do"], a["ds"],
                 a["dq"], a["dk"], a["dv"], a["d0"], a["ws"], a["nws"], a["B"], a["H"], a["T"], a["K"], a["V"],
                 a["dt"], None)

    for name in ("q", "k", "v", "g", "do", "dq", "dk", "dv", "d0"):
        assert call(**{name: None}) == NULL, name
    for kw, status in ((dict(dt=-1), DTYPE), (dict(V=7), SHAPE), (dict(q=P(q.value + 8)), ALIGN),
                       (dict(q=P(q.value + 4), qs=qs, ks=ks, vs=vs), ALIGN), (dict(qs=qs), NULL),
                       (dict(ks=ks, vs=vs), NULL), (dict(do=P(do.value + 2)), ALIGN),
                       (dict(ws=None), WORKSPACE), (dict(nws=64), WORKSPACE), (dict(dq=q), ALIAS), (dict(dk=do), ALIAS),
                       (dict(dv=dk), ALIAS), (dict(d0=ds), ALIAS), (dict(d0=s0), ALIAS), (dict(dq=qs, qs=qs, ks=ks, vs=vs), ALIAS),
                       (dict(ws=dq), ALIAS), (dict(ws=vs, qs=qs, ks=ks, vs=vs), ALIAS), (dict(dk=g), ALIAS)):
        assert call(**kw) == status, kw


@cpu_only
def test_layer_norm_refusals():
    lib = _lib.load()
    x, w, b, y, m, r, dy, dx, dw, db, ws, xs = (_at(i) for i in range(12))

    def fwd(x=x, w=w, b=b, eps=1e-5, y=y, m=m, r=r, B=1, H=2, T=5, D=16, dt=BF16):
        return lib.kda_layer_norm_fwd(x, w, b, eps, y, m, r, B, H, T, D, dt, None)

    for kw, status in ((dict(x=None), NULL), (dict(y=None), NULL), (dict(dt=9), DTYPE), (dict(D=0), SHAPE),
                       (dict(T=-1), SHAPE), (dict(B=0), SHAPE), (dict(eps=-1.0), SHAPE), (dict(eps=float("nan")), SHAPE),
                       (dict(eps=float("inf")), SHAPE), (dict(T=1 << 30), SHAPE),
                       (dict(B=1 << 11, H=1 << 10), SHAPE), (dict(H=1 << 16, D=1 << 13), SHAPE), (dict(x=P(x.value + 1)), ALIGN),
                       (dict(y=P(y.value + 2), dt=F32), ALIGN), (dict(y=x), ALIAS), (dict(y=w), ALIAS),
                       (dict(m=x), ALIAS), (dict(m=r), ALIAS), (dict(r=y), ALIAS)):
        assert fwd(**kw) == status, kw

    def bwd(x=x, xs=None, w=w, m=m, r=r, dy=dy, dx=dx, dw=dw, db=db, ws=ws, nws=1 << 20, B=1, H=2, T=5, D=64, dt=BF16):
        return lib.kda_layer_norm_bwd(x, xs, w, m, r, dy, dx, dw, db, ws, nws, B, H, T, D, dt, None)

    for name in ("x", "m", "r", "dy", "dx"):
        assert bwd(**{name: None}) == NULL, name
    for kw, status in ((dict(dt=9), DTYPE), (dict(D=0), SHAPE), (dict(D=40, xs=xs), SHAPE), (dict(ws=None), WORKSPACE),
                       (dict(nws=8), WORKSPACE), (dict(ws=P(ws.value + 4)), ALIGN), (dict(dx=P(dx.value + 1)), ALIGN),
                       (dict(dx=x), ALIAS), (dict(dx=P(dy.value + 2)), ALIAS), (dict(dw=dx), ALIAS), (dict(db=dw), ALIAS),
                       (dict(dw=m), ALIAS), (dict(ws=dx), ALIAS), (dict(ws=xs, xs=xs), ALIAS)):
        assert bwd(**kw) == status, kw


@cpu_only
def test_ckpt_refusals():
    lib = _lib.load()
    x, c, s = (_at(i) for i in range(3))
    for fn, order in ((lib.kda_ckpt_pack, lambda x, c, s: (x, c, s)), (lib.kda_ckpt_unpack, lambda x, c, s: (c, s, x))):
        def call(x=x, c=c, s=s, rows=4, D=64, dt=BF16):
            return fn(*order(x, c, s), rows, D, dt, None)

        for kw, status in ((dict(x=None), NULL), (dict(c=None), NULL), (dict(s=None), NULL), (dict(dt=4), DTYPE),
                           (dict(D=0), SHAPE), (dict(D=33), SHAPE), (dict(rows=-1), SHAPE), (dict(rows=1 << 50), SHAPE),
                           (dict(x=P(x.value + 1)), ALIGN), (dict(c=x), ALIAS), (dict(s=c), ALIAS),
                           (dict(s=P(x.value + 64)), ALIAS)):
            assert call(**kw) == status, kw


def test_binding_refuses_before_the_library():
    f32 = torch.float32
    q, v, g = torch.zeros(1, 2, 4, 8), torch.zeros(1, 2, 4, 8), torch.zeros(2)
    with pytest.raises(ValueError):                              # not on the GPU
        kda.decay_attn_step(q[:, :, 0].contiguous(), q[:, :, 0].contiguous(), v[:, :, 0].contiguous(), g,
                            torch.zeros(1, 2, 8, 8))
    for kw, err in ((dict(k=q.bfloat16()), TypeError), (dict(k=q[:, :, :3]), ValueError),
                    (dict(log_decay=torch.zeros(3)), ValueError), (dict(log_decay=g.double()), TypeError),
                    (dict(state_in=torch.zeros(1, 2, 8, 4)), ValueError), (dict(lengths=torch.zeros(1)), TypeError),
                    (dict(lengths=torch.zeros(2, dtype=torch.int32)), ValueError),
                    (dict(out=torch.zeros(1, 2, 3, 8)), ValueError), (dict(q=q.half(), k=q.half(), v=q.half()), TypeError)):
        a = {**dict(q=q, k=q, v=v, log_decay=g), **kw}
        with pytest.raises(err):
            kda.decay_attn_fwd(**a)
    codes, scales = torch.zeros(1, 2, 4, 8, dtype=torch.uint8), torch.zeros(1, 2, 4, 1, dtype=torch.uint8)
    for bad in ((codes, scales[..., 0]), (codes.to(f32), scales), (codes[:, :1], scales), (codes, scales)):
        with pytest.raises((ValueError, TypeError)):
            kda.decay_attn_bwd(q, bad, v, g, None, v)
    with pytest.raises(TypeError):
        kda.layer_norm_bwd(q, None, None, torch.zeros(1, 2, 4), q)
    with pytest.raises(ValueError):
        kda.ckpt_unpack(codes, torch.zeros(1, 2, 4, 2, dtype=torch.uint8))
    with pytest.raises(TypeError):
        kda.ckpt_pack(q.half())
