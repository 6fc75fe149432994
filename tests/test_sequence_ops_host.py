"""Refusals of the short convolution, the query and key norm with rotation and the gated recurrence (every argument
error is reported before anything is launched: these calls pass fake device addresses, so they run only where no GPU is
visible), and the host-only frequencies."""
import ctypes

import numpy as np
import pytest
import torch

import gated_delta_rule_47_amd as kda
from gated_delta_rule_47_amd import _lib
from oracle import sequence_ref as R


def _gpu_visible():
    try:
        return torch.cuda.is_available()
    except Exception:
        return False


cpu_only = pytest.mark.skipif(_gpu_visible(), reason="fake device pointers: CPU-only check")
P = ctypes.c_void_p
NULL, SHAPE, DTYPE, ALIAS, HIP, WORKSPACE, ALIGN = -1, -2, -3, -5, -6, -7, -8
F32, BF16 = 0, 1


def _at(i):
    return P(0x10000000 * (i + 1))


def _off(p, n):
    return P(p.value + n)


def _run(fn, order, ok, cases):
    before = kda.counters()["rejected"]
    for kw, status in cases:
        a = {**ok, **kw}
        assert fn(*(a[n] for n in order), None) == status, kw
    assert kda.counters()["rejected"] - before == len(cases)


def test_chunk_constant_is_the_header_s():
    import os
    text = open(os.path.join(os.path.dirname(__file__), "..", "include", "kda.h")).read()
    assert "#define KDA_GATED_SCAN_CHUNK %d\n" % kda.GATED_SCAN_CHUNK in text


def test_workspace_bytes():
    lib = _lib.load()
    f, b = lib.kda_gated_scan_workspace_bytes, lib.kda_gated_scan_bwd_workspace_bytes
    assert f(1, 8, 64, 64, F32) == 0 and f(1, 8, 0, 64, F32) == 0 and f(1, 1, 30011, 4096, BF16) > 0
    assert b(1, 8, 32, 64, F32) >= 8 * 64 * 8 and b(1, 1, 1 << 14, 4096, BF16) > b(1, 1, 1 << 13, 4096, BF16)
    for args in ((0, 1, 64, 64, F32), (1, 0, 64, 64, F32), (1, 1, -1, 64, F32), (1, 1, 64, 0, F32), (1, 1, 64, 64, 5),
                 (1, 1, (1 << 28) + 1, 1, F32), (1, 2, 1 << 28, 64, F32), (1, 1, 1, (1 << 26) + 1, F32), (1 << 11, 1 << 10, 1, 1, F32)):
        assert f(*args) == 0 and b(*args) == 0, args
    c = lib.kda_short_conv_bwd_workspace_bytes
    assert c(8, 8, 4096, 64, 4, BF16) % (512 * 5 * 4) == 0 and c(8, 8, 4096, 64, 4, BF16) > 0
    for args in ((1, 1, 4, 12, 4, F32), (1, 1, 4, 16, 1, F32), (1, 1, 4, 16, 5, F32), (0, 1, 4, 16, 4, F32),
                 (1, 1, 4, 16, 4, 2), (1, 1, (1 << 28) + 1, 16, 4, F32), (1, 2, 4, 1 << 20, 4, F32)):
        assert c(*args) == 0, args
    q = lib.kda_qk_norm_rope_bwd_workspace_bytes
    assert q(1, 128, 4, 1, 4, 1, 64) % 256 == 0 and q(1, 128, 4, 1, 4, 1, 64) > 0 and q(1, 128, 4, 4, 0, 1, 64) > 0
    for args in ((1, 128, 4, 2, 4, 1, 64), (1, 128, 0, 1, 0, 1, 64), (1, 128, 4, 1, 4, 1, 264), (1, 128, 4, 1, 4, 1, 60),
                 (1 << 16, 1 << 16, 4, 1, 4, 1, 64), (1, 128, 1 << 15, 1, 4, 1, 64)):
        assert q(*args) == 0, args


@cpu_only
def test_short_conv_refusals():
    lib = _lib.load()
    x, w, b, n, s, y, e = (_at(i) for i in range(7))
    order = "x xb xt w b n s act y e B H T D W dt".split()
    ok = dict(x=x, xb=64 * 16, xt=16, w=w, b=b, n=n, s=s, act=1, y=y, e=e, B=2, H=2, T=64, D=8, W=4, dt=BF16)
    _run(lib.kda_short_conv_fwd, order, ok, [
        (dict(x=None), NULL), (dict(w=None), NULL), (dict(y=None), NULL), (dict(dt=3), DTYPE), (dict(B=0), SHAPE),
        (dict(H=0), SHAPE), (dict(T=-1), SHAPE), (dict(D=12), SHAPE), (dict(D=0), SHAPE), (dict(W=1), SHAPE), (dict(W=5), SHAPE),
        (dict(act=2), SHAPE), (dict(act=-1), SHAPE), (dict(xt=-16), SHAPE), (dict(xb=-1), SHAPE), (dict(xt=1 << 46), SHAPE),
        (dict(T=(1 << 28) + 1), SHAPE), (dict(H=1 << 18), SHAPE), (dict(B=(1 << 20) + 1), SHAPE), (dict(x=_off(x, 1)), ALIGN),
        (dict(y=_off(y, 1)), ALIGN), (dict(w=_off(w, 2)), ALIGN), (dict(b=_off(b, 2)), ALIGN), (dict(n=_off(n, 2)), ALIGN),
        (dict(s=_off(s, 1)), ALIGN), (dict(y=x), ALIAS), (dict(y=_off(x, 2 * 64 * 16 * 2 - 2)), ALIAS), (dict(y=w), ALIAS),
        (dict(e=s), ALIAS), (dict(e=y), ALIAS), (dict(e=x), ALIAS), (dict(y=n), ALIAS), (dict(y=b), ALIAS)])
    order = "x xb w b act s y B H D W dt".split()
    ok = dict(x=x, xb=16, w=w, b=b, act=0, s=s, y=y, B=2, H=2, D=8, W=4, dt=F32)
    _run(lib.kda_short_conv_step, order, ok, [
        (dict(x=None), NULL), (dict(w=None), NULL), (dict(s=None), NULL), (dict(y=None), NULL), (dict(dt=3), DTYPE),
        (dict(D=4), SHAPE), (dict(W=7), SHAPE), (dict(act=9), SHAPE), (dict(xb=-16), SHAPE), (dict(y=_off(y, 2)), ALIGN),
        (dict(s=_off(s, 2)), ALIGN), (dict(y=x), ALIAS), (dict(y=s), ALIAS), (dict(s=x), ALIAS), (dict(s=w), ALIAS)])
    dy, ds, dx, dw, db, d0, ws = (_at(i + 7) for i in range(7))
    order = "x xb xt w b n s act dy ds dx db_ dt_ dw db d0 ws nws B H T D W dt".split()
    ok = dict(x=x, xb=64 * 16, xt=16, w=w, b=b, n=n, s=s, act=1, dy=dy, ds=ds, dx=dx, db_=64 * 16, dt_=16, dw=dw, db=db, d0=d0,
              ws=ws, nws=1 << 20, B=2, H=2, T=64, D=8, W=4, dt=BF16)
    _run(lib.kda_short_conv_bwd, order, ok, [
        (dict(x=None), NULL), (dict(w=None), NULL), (dict(dy=None), NULL), (dict(dx=None), NULL), (dict(d0=None), NULL),
        (dict(dt=-1), DTYPE), (dict(W=0), SHAPE), (dict(act=3), SHAPE), (dict(dt_=15), SHAPE), (dict(dt_=0), SHAPE),
        (dict(db_=64 * 16 - 1), SHAPE), (dict(dt_=16, db_=8), SHAPE), (dict(ws=None), WORKSPACE), (dict(nws=12), WORKSPACE),
        (dict(ws=_off(ws, 8)), ALIGN), (dict(dx=_off(dx, 1)), ALIGN), (dict(dw=_off(dw, 1)), ALIGN), (dict(dx=x), ALIAS),
        (dict(dx=dy), ALIAS), (dict(dw=w), ALIAS), (dict(db=dw), ALIAS), (dict(d0=ds), ALIAS), (dict(d0=s), ALIAS),
        (dict(ws=dx), ALIAS), (dict(ws=n), ALIAS),
        # a slice next to x's own rows in one wide buffer may not reach into them
        (dict(xt=32, xb=64 * 32, dx=_off(x, 31), dt_=32, db_=64 * 32, dt=F32), ALIGN),
        (dict(xt=32, xb=64 * 32, dx=_off(x, 60), dt_=32, db_=64 * 32, dt=F32), ALIAS),
        (dict(xt=32, xb=64 * 32, dx=_off(x, 68), dt_=32, db_=64 * 32, dt=F32), ALIAS),
        (dict(xt=32, xb=64 * 32, dx=_off(x, 64), dt_=31, db_=64 * 31, dt=F32), ALIAS),
        # (beside them it passes every check: without a GPU the launch fails)
        (dict(xt=32, xb=64 * 32, dx=_off(x, 64), dt_=32, db_=64 * 32, dt=F32), HIP),
        (dict(xt=2 * 32, xb=32, dx=_off(x, 64), dt_=2 * 32, db_=32, dt=F32), HIP)])


@cpu_only
def test_qk_refusals():
    lib = _lib.load()
    q, k, qw, kw, f, p, yq, yk = (_at(i) for i in range(8))
    order = "q qb qt qh k kb kt kh qw Hqw kw Hkw norm eps f p scale inter yq yk B T Hq Hk D R dt".split()
    n = 8 * 32                                     # channels of the fused projection: 4 + 2 + 2 heads of 32
    ok = dict(q=q, qb=16 * n, qt=n, qh=32, k=k, kb=16 * n, kt=n, kh=32, qw=qw, Hqw=1, kw=kw, Hkw=1, norm=1, eps=1e-6, f=f, p=p,
              scale=1.0, inter=0, yq=yq, yk=yk, B=2, T=16, Hq=4, Hk=2, D=32, R=32, dt=BF16)
    shared = [
        (dict(f=None), NULL), (dict(dt=2), DTYPE), (dict(B=0), SHAPE), (dict(T=-1), SHAPE), (dict(Hq=-1), SHAPE),
        (dict(Hq=0, Hk=0), SHAPE), (dict(D=36), SHAPE), (dict(D=264, R=0), SHAPE), (dict(D=0, R=0), SHAPE), (dict(R=36), SHAPE),
        (dict(R=40), SHAPE), (dict(R=-8), SHAPE), (dict(Hqw=2), SHAPE), (dict(Hkw=4), SHAPE), (dict(norm=3), SHAPE),
        (dict(norm=-1), SHAPE), (dict(norm=0), SHAPE), (dict(eps=-1e-6), SHAPE), (dict(eps=float("nan")), SHAPE),
        (dict(eps=float("inf")), SHAPE), (dict(scale=float("nan")), SHAPE), (dict(scale=float("inf")), SHAPE), (dict(qh=-32), SHAPE),
        (dict(kt=-1), SHAPE), (dict(qt=1 << 47), SHAPE), (dict(B=1 << 16, T=1 << 16), SHAPE), (dict(q=_off(q, 1)), ALIGN),
        (dict(f=_off(f, 4)), ALIGN), (dict(p=_off(p, 2)), ALIGN), (dict(qw=_off(qw, 2)), ALIGN)]
    _run(lib.kda_qk_norm_rope_fwd, order, ok, shared + [
        (dict(q=None), NULL), (dict(k=None), NULL), (dict(yq=None), NULL), (dict(yk=None), NULL), (dict(yk=_off(yk, 1)), ALIGN),
        (dict(yq=q), ALIAS), (dict(yq=_off(k, 64)), ALIAS), (dict(yk=yq), ALIAS), (dict(yk=qw), ALIAS), (dict(yq=f), ALIAS),
        (dict(yq=p), ALIAS)])
    dq_, dk_, dq, dk, gq, gk, ws = (_at(i + 8) for i in range(7))
    dk = _off(dq, 4 * 32 * 2)                      # next to dq in one fused gradient
    order = ("q qb qt qh k kb kt kh qw Hqw kw Hkw norm eps f p scale inter dq_ dk_ dq oqb oqt oqh dk okb okt okh gq gk ws nws "
             "B T Hq Hk D R dt").split()
    ok = dict(ok, dq_=dq_, dk_=dk_, dq=dq, oqb=16 * n, oqt=n, oqh=32, dk=dk, okb=16 * n, okt=n, okh=32, gq=gq, gk=gk, ws=ws,
              nws=1 << 20)
    _run(lib.kda_qk_norm_rope_bwd, order, ok, shared + [
        (dict(q=None), NULL), (dict(k=None), NULL), (dict(dq_=None), NULL), (dict(dk_=None), NULL), (dict(dq=None), NULL),
        (dict(dk=None), NULL), (dict(norm=0, qw=None, kw=None), SHAPE), (dict(Hk=0, kw=None), SHAPE), (dict(oqh=31), SHAPE),
        (dict(oqt=n // 2 - 1), SHAPE), (dict(oqb=0), SHAPE), (dict(okt=0), SHAPE), (dict(ws=None), WORKSPACE), (dict(nws=8), WORKSPACE),
        (dict(ws=_off(ws, 4)), ALIGN), (dict(dq=_off(dq, 1)), ALIGN), (dict(dk=_off(dk, -2)), ALIAS), (dict(dk=dq), ALIAS),
        (dict(dk=_off(dq, 7 * 32 * 2)), ALIAS), (dict(dq=q), ALIAS), (dict(dq=dq_), ALIAS), (dict(gq=qw), ALIAS), (dict(gk=gq), ALIAS),
        (dict(ws=dk), ALIAS), (dict(ws=p), ALIAS), ({}, HIP)])


@cpu_only
def test_gated_scan_refusals():
    lib = _lib.load()
    x, z, A, b, i, n, s, y, e, c, ws = (_at(i) for i in range(11))
    order = "x z A b i n s norm y e c ws nws B H T D dt".split()
    ok = dict(x=x, z=z, A=A, b=b, i=i, n=n, s=s, norm=1, y=y, e=e, c=c, ws=ws, nws=1 << 26, B=2, H=3, T=600, D=16, dt=BF16)
    shared = [(dict(x=None), NULL), (dict(z=None), NULL), (dict(A=None), NULL), (dict(dt=7), DTYPE), (dict(B=0), SHAPE),
              (dict(H=0), SHAPE), (dict(D=0), SHAPE), (dict(x=_off(x, 1)), ALIGN), (dict(i=_off(i, 1)), ALIGN),
              (dict(A=_off(A, 2)), ALIGN), (dict(b=_off(b, 1)), ALIGN)]
    time = [(dict(T=-1), SHAPE), (dict(T=(1 << 28) + 1), SHAPE), (dict(T=1 << 28, D=64), SHAPE), (dict(ws=None), WORKSPACE),
            (dict(nws=64), WORKSPACE), (dict(ws=_off(ws, 128)), ALIGN), (dict(n=_off(n, 1)), ALIGN), (dict(c=_off(c, 2)), ALIGN)]
    _run(lib.kda_gated_scan_fwd, order, ok, shared + time + [
        (dict(y=None), NULL), (dict(y=x), ALIAS), (dict(y=_off(z, 2)), ALIAS), (dict(y=i), ALIAS), (dict(e=b), ALIAS), (dict(e=y), ALIAS),
        (dict(e=_off(s, 4)), ALIAS), (dict(c=s), ALIAS), (dict(c=e), ALIAS), (dict(ws=y), ALIAS), (dict(ws=n), ALIAS), (dict(y=A), ALIAS),
        (dict(e=_off(e, 2)), ALIGN), (dict(s=_off(s, 2)), ALIGN)])
    order = "x z A b i norm s y B H D dt".split()
    _run(lib.kda_gated_scan_step, order, ok, shared + [
        (dict(s=None), NULL), (dict(y=None), NULL), (dict(s=x), ALIAS), (dict(y=s), ALIAS), (dict(y=z), ALIAS), (dict(s=_off(s, 2)), ALIGN),
        (dict(s=A), ALIAS), (dict(s=b), ALIAS), (dict(y=i), ALIAS)])
    dy, ds, dx, dz, di, dA, db, d0 = (_at(i + 11) for i in range(8))
    order = "x z A b i n norm c dy ds dx dz di dA db d0 ws nws B H T D dt".split()
    ok = dict(ok, dy=dy, ds=ds, dx=dx, dz=dz, di=di, dA=dA, db=db, d0=d0)
    _run(lib.kda_gated_scan_bwd, order, ok, shared + time + [
        (dict(c=None), NULL), (dict(dy=None), NULL), (dict(dx=None), NULL), (dict(dz=None), NULL), (dict(d0=None), NULL),
        (dict(di=None), NULL), (dict(i=None), NULL), (dict(dx=x), ALIAS), (dict(dx=dy), ALIAS), (dict(dz=dx), ALIAS), (dict(di=z), ALIAS),
        (dict(dA=A), ALIAS), (dict(db=b), ALIAS), (dict(d0=ds), ALIAS), (dict(d0=c), ALIAS), (dict(ws=dz), ALIAS), (dict(dy=_off(dy, 1)), ALIGN),
        (dict(dA=_off(dA, 1)), ALIGN)])


@pytest.mark.parametrize("R_", [2, 8, 64, 96, 128])
@pytest.mark.parametrize("scaling,kw", [(None, {}), ("linear", dict(factor=4.0)), ("base", dict(factor=8.0)), ("parts", dict(factor=1.0)),
                                        ("parts", dict(factor=8.0)), ("parts", dict(factor=40.0, trained_length=65536, base=5e5)),
                                        ("parts", dict(factor=16.0, trained_length=128, fast_turns=8.0, slow_turns=2.0))])
def test_rope_frequencies(R_, scaling, kw):
    """Each value is a power and a few products: 1e-13 is over a thousand roundings of 2^-53, times the logarithm of the
    base in the exponent."""
    if scaling == "base" and R_ == 2:
        with pytest.raises(kda.KdaError):
            kda.rope_frequencies(R_, scaling=scaling, **kw)
        return
    f, s = kda.rope_frequencies(R_, scaling=scaling, **kw)
    names = {"trained_length": "trained", "fast_turns": "fast", "slow_turns": "slow"}
    rf, rs = R.rope_frequencies(R_, scaling=scaling, **{names.get(k, k): v for k, v in kw.items()})
    assert f.dtype == torch.float64 and f.shape == (R_ // 2,)
    assert np.allclose(f.numpy(), rf, rtol=1e-13, atol=0) and abs(s - rs) <= 1e-13
    base = kw.get("base", 10000.0)
    plain = base ** (-np.arange(0, R_, 2) / R_)
    factor = kw.get("factor", 1.0)
    assert np.all(f.numpy() <= plain * (1 + 1e-13)) and np.all(f.numpy() >= plain / factor * (1 - 1e-13))
    if scaling == "base":                          # the slowest pair slowed by the whole factor, the fastest left
        assert abs(f[-1] / (plain[-1] / factor) - 1) < 1e-12 and f[0] == 1


def test_rope_frequencies_refusals():
    for kw in (dict(rot_dim=0), dict(rot_dim=7), dict(rot_dim=-2), dict(base=1.0), dict(base=float("nan")), dict(factor=0.5),
               dict(factor=float("inf")), dict(scaling="parts", trained_length=0), dict(scaling="parts", slow_turns=0.0),
               dict(scaling="parts", fast_turns=1.0), dict(scaling="base", factor=1e200, rot_dim=4)):
        with pytest.raises(kda.KdaError) as e:
            kda.rope_frequencies(**{"rot_dim": 8, **kw})
        assert e.value.status == SHAPE, kw
    with pytest.raises(ValueError):
        kda.rope_frequencies(8, scaling="other")
    lib = _lib.load()
    d = ctypes.c_double()
    assert lib.kda_rope_frequencies(None, ctypes.byref(d), 8, 1e4, 0, 1.0, 1.0, 32.0, 1.0) == NULL
    assert lib.kda_rope_frequencies(ctypes.byref(d), ctypes.byref(d), 8, 1e4, 4, 1.0, 1.0, 32.0, 1.0) == SHAPE


def test_binding_refuses_before_the_library():
    x, w = torch.zeros(2, 5, 16), torch.zeros(16, 4)
    with pytest.raises(ValueError):                              # not on the GPU
        kda.short_conv_fwd(x, w)
    for kw, err in ((dict(weight=torch.zeros(8, 4)), ValueError), (dict(weight=w.double()), TypeError), (dict(heads=3), ValueError),
                    (dict(heads=0), ValueError), (dict(activation="relu"), ValueError), (dict(state_in=torch.zeros(2, 4, 16)), ValueError),
                    (dict(state_in=torch.zeros(2, 3, 16).bfloat16()), TypeError), (dict(lengths=torch.zeros(2)), TypeError),
                    (dict(x=x.half()), TypeError), (dict(x=torch.zeros(2, 5, 32)[..., ::2]), ValueError),
                    (dict(out=torch.zeros(2, 1, 5, 15)), ValueError), (dict(bias=torch.zeros(4)), ValueError)):
        with pytest.raises(err):
            kda.short_conv_fwd(**{**dict(x=x, weight=w), **kw})
    with pytest.raises(ValueError):
        kda.short_conv_bwd(x, w, None, None, torch.zeros(2, 3, 5, 5))
    q, f = torch.zeros(2, 5, 4, 16), torch.zeros(8, dtype=torch.float64)
    for kw, err in ((dict(k=torch.zeros(2, 4, 4, 16)), ValueError), (dict(k=q.bfloat16()), TypeError), (dict(freqs=f.float()), TypeError),
                    (dict(positions=torch.zeros(2, 5)), TypeError), (dict(positions=torch.zeros(5, dtype=torch.int32)), ValueError),
                    (dict(q_weight=torch.zeros(2, 16)), ValueError), (dict(q_weight=torch.zeros(1, 8)), ValueError),
                    (dict(k=None, k_weight=torch.zeros(1, 16)), ValueError), (dict(norm="layer"), ValueError),
                    (dict(q_out=torch.zeros(2, 5, 4, 16)), ValueError), (dict(q=torch.zeros(2, 5, 16, 4).transpose(2, 3)), ValueError)):
        with pytest.raises(err):
            kda.qk_norm_rope_fwd(**{**dict(q=q, k=q, freqs=f), **kw})
    g = torch.zeros(2, 3, 40, 8)
    for kw, err in ((dict(z=g[:, :, :39]), ValueError), (dict(z=g.bfloat16()), TypeError), (dict(A_log=torch.zeros(2)), ValueError),
                    (dict(dt_bias=torch.zeros(3)), ValueError), (dict(input_gate=g.double()), TypeError),
                    (dict(state_in=torch.zeros(2, 3, 4)), ValueError), (dict(x=g.transpose(2, 3), z=g.transpose(2, 3)), ValueError)):
        with pytest.raises(err):
            kda.gated_scan_fwd(**{**dict(x=g, z=g, A_log=torch.zeros(3)), **kw})
    with pytest.raises(ValueError):                              # one chunk's state too few
        kda.gated_scan_bwd(g, g, torch.zeros(3), None, torch.zeros(2, 3, 1, 8), g)


def test_sizes_of_more_than_32_bits():
    """A size that 32 bits would cut to a small one is refused (an expanded tensor holds it in little memory)."""
    far = (1 << 32) + 16
    e = lambda *s: torch.zeros((1,) * (len(s) - 1) + (s[-1],)).expand(*s)
    w, f, A, one = torch.zeros(16, 4), torch.zeros(8, dtype=torch.float64), torch.zeros(1), torch.zeros(1, 2, 1, 16)
    for call in (lambda: kda.short_conv_fwd(e(1, far, 16), w), lambda: kda.short_conv_fwd(e(far, 0, 16), w),
                 lambda: kda.short_conv_fwd(e(1, 2, 16), torch.zeros(1, 1).expand(16, far)),
                 lambda: kda.short_conv_step(e(far, 16), w, None, torch.zeros(1, 3, 16)),
                 lambda: kda.short_conv_bwd(e(1, far, 16), w, None, None, e(1, 1, far, 16)),
                 lambda: kda.qk_norm_rope_fwd(e(1, far, 1, 16), None, f), lambda: kda.qk_norm_rope_fwd(one, e(1, 2, far, 16), f),
                 lambda: kda.qk_norm_rope_fwd(one, None, torch.zeros(1, dtype=torch.float64).expand(far // 2)),
                 lambda: kda.qk_norm_rope_bwd(e(far, 1, 1, 16), None, f, None, None),
                 lambda: kda.gated_scan_fwd(e(1, 1, far, 16), e(1, 1, far, 16), A),
                 lambda: kda.gated_scan_step(e(1, far, 16), e(1, far, 16), A, None, None),
                 lambda: kda.gated_scan_bwd(e(1, 1, far, 16), e(1, 1, far, 16), A, None, None, None),
                 lambda: kda.gated_scan_workspace_bytes(1, 1, far, 16), lambda: kda.gated_scan_bwd_workspace_bytes(far, 1, 1, 16),
                 lambda: kda.short_conv_bwd_workspace_bytes(1, 1, far, 16, 4),
                 lambda: kda.qk_norm_rope_bwd_workspace_bytes(1, far, 1, 1, 16),
                 lambda: kda.rope_frequencies(far)):
        with pytest.raises(kda.KdaError) as err:
            call()
        assert err.value.status == SHAPE


@pytest.mark.parametrize("R_,base,trained,factor", [(128, 1e4, 65536, 8.0), (128, 1e4, 131072, 8.0), (128, 1e4, 262144, 8.0), (64, 1e4, 1 << 20, 40.0),
                                                    (8, 500.0, 32768, 4.0), (2, 1e4, 4096, 8.0), (96, 5e5, 8192, 16.0)])
def test_rotation_by_parts_in_turns(R_, base, trained, factor):
    """The rule as it is stated: pairs of more than fast_turns turns over the trained length are left, only those below
    slow_turns take the whole factor, and between the last whole pair in front of the ramp and the first behind it, which may
    stand behind the table, the share grows by the same step from pair to pair."""
    fast, slow = 32.0, 1.0
    f = kda.rope_frequencies(R_, base, "parts", factor, trained, fast, slow)[0].numpy()
    turns = lambda p: base ** (-2.0 * p / R_) * trained / (2 * np.pi)
    first = max(p for p in range(R_) if turns(p) >= fast)
    behind = min(p for p in range(R_) if turns(p) <= slow)
    assert first >= 0 and behind < R_ - 1 or R_ == 2
    for p in range(R_ // 2):
        slowed = turns(p) * 2 * np.pi / trained / f[p]
        share = min(max((p - first) / (behind - first), 0.0), 1.0)
        # 1 - share (1 - 1 / factor): a few roundings of 2^-53 times the exponent's logarithm, as above
        assert abs(1 / slowed - (1 - share * (1 - 1 / factor))) <= 1e-13, p
        if turns(p) >= fast:
            assert abs(slowed - 1) <= 1e-13, p
        if turns(p) > slow:
            assert slowed < factor * (1 - 1e-6), p
    rf, _ = R.rope_frequencies(R_, base, "parts", factor, trained)
    assert np.allclose(f, rf, rtol=1e-13, atol=0)
