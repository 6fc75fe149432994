"""Layer norm forward and backward on the GPU against float64.

Tolerances: one rounding to bf16 is off by at most u = 2^-8 of the value (fp32: 2^-24).  The fp32 sums
over a row of D run in at most D / 64 + 14 additions per lane and tree, the sums over rows of the
weight's gradient in at most a few hundred: 1000 2^-24 = 6e-5 of the sums over absolute values bounds
them all; in the 2-norm, with roundings that do not line up, 2e-5 is asked for.
"""
import numpy as np
import pytest
import torch

import gated_delta_rule_47_amd as kda
from oracle import layer_ref as R

from gpu_helpers import DEV, host, say, to_dev

pytestmark = pytest.mark.gpu
U = 2.0 ** -8
F32 = 2e-5
BF, FP = torch.bfloat16, torch.float32


def norm2(got, ref):
    n = np.linalg.norm(ref)
    return np.linalg.norm(got - ref) / n if n else float(np.abs(got).max(initial=0.0))


def run(B, H, T, D, dtype, params=True, shift=0, packed=False, seed=0, offset=0.0):
    """shift: elements by which the tensors' storage is moved off its alignment."""
    say("norm", B, H, T, D, dtype, params, shift, packed)
    rng = np.random.default_rng(seed)

    def moved(a):
        t = to_dev(a, dtype)
        buf = torch.empty(t.numel() + shift, dtype=dtype, device=DEV)[shift:].view(t.shape)
        return buf.copy_(t)

    xd = moved((offset + rng.standard_normal((B, H, T, D)) * np.exp(rng.standard_normal((B, H, T, 1)))).astype(np.float32))
    dyd = moved(rng.standard_normal((B, H, T, D)).astype(np.float32))
    w = b = wd = bd = None
    if params:
        w = (1 + 0.3 * rng.standard_normal((H, D))).astype(np.float32)
        b = rng.standard_normal((H, D)).astype(np.float32)
        wd, bd = to_dev(w, FP), to_dev(b, FP)
    x, dy = host(xd), host(dyd)
    y, mean, rstd = kda.layer_norm_fwd(xd, wd, bd, out=moved(np.zeros((B, H, T, D), np.float32)))
    torch.cuda.synchronize()
    ry, rm, rr = R.layer_norm(x, w, b)
    bar = U if dtype == BF else F32
    assert norm2(host(y), ry) <= bar
    assert np.abs(host(mean) - rm).max(initial=0) <= F32 * np.abs(x).max(initial=1.0)
    assert norm2(host(rstd), rr) <= F32
    xarg = xd
    if packed:
        xarg = kda.ckpt_pack(xd)
        x = R.ckpt_unpack(*(t.cpu().numpy() for t in xarg))
    dx, dw, db = kda.layer_norm_bwd(xarg, wd, mean, rstd, dyd)
    torch.cuda.synchronize()
    rdx, rdw, rdb = R.layer_norm_adjoint(x, w, host(mean), host(rstd), dy)
    # dx is a difference of terms of the size of rstd p: its error is measured against those (a row of
    # one element has dx = 0)
    p = np.abs(dy if w is None else dy * w[None, :, None].astype(np.float64))
    xh = np.abs((x - host(mean)[..., None]) * host(rstd)[..., None])
    M = host(rstd)[..., None] * (p + p.mean(-1, keepdims=True) + xh * (p * xh).mean(-1, keepdims=True))
    lim = (1.05 * U * np.abs(rdx) if dtype == BF else 0) + 1000 * 2.0 ** -24 * M
    assert np.all(np.abs(host(dx) - rdx) <= lim)
    for name, got, ref, mag in (("dw", dw, rdw, (np.abs(dy) * xh).sum((0, 2))), ("db", db, rdb, np.abs(dy).sum((0, 2)))):
        assert np.all(np.abs(host(got) - ref) <= 1000 * 2.0 ** -24 * mag + 1e-30), name
        assert np.linalg.norm(host(got) - ref) <= F32 * np.linalg.norm(mag) / 4, name


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("D", [1, 2, 3, 7, 8, 9, 16, 24, 32, 33, 63, 64, 65, 96, 128, 200, 256, 257, 512, 640, 1000,
                               1024, 1025, 2048, 2055, 4096, 4104, 5001, 8192, 8200, 16384, 16392, 20001])
def test_widths(D, dtype):
    run(1, 2, 5, D, dtype, seed=D)


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("D", [32, 96, 128, 512, 1000])
def test_rows_off_their_alignment(D, dtype):
    run(2, 1, 7, D, dtype, shift=1)
    run(2, 1, 7, D, dtype, shift=2, params=False)


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("B,H,T", [(1, 1, 1), (3, 4, 1), (2, 3, 63), (1, 5, 300), (2, 1, 5000), (40, 70, 3)])
def test_rows(B, H, T, dtype):
    run(B, H, T, 64, dtype, seed=T)
    run(B, H, T, 65, dtype, seed=T, params=False)


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("D", [8, 24, 32, 64, 128, 512, 4096, 16416])
def test_bwd_from_8_bits(D, dtype):
    run(2, 2, 40 if D < 4096 else 3, D, dtype, packed=True)


def test_far_from_zero():
    run(1, 2, 50, 128, FP, offset=300.0)


def test_constant_rows_and_non_finite():
    x = torch.full((1, 1, 4, 64), 3.0, device=DEV)
    x[0, 0, 2, 5] = float("nan")
    x[0, 0, 3, 5] = float("inf")
    y, mean, rstd = kda.layer_norm_fwd(x, eps=1e-5)
    assert torch.all(y[0, 0, :2] == 0) and torch.all(mean[0, 0, :2] == 3.0)
    assert torch.allclose(rstd[0, 0, :2], torch.tensor(1e-5, device=DEV).rsqrt())
    assert torch.all(torch.isnan(y[0, 0, 2:])) and torch.all(torch.isnan(rstd[0, 0, 2:]))   # rows keep to themselves
    assert torch.all(torch.isnan(kda.layer_norm_fwd(x[:, :, :1].contiguous(), eps=0.0)[0]))   # 0 / 0, as the formula


def test_options_and_no_rows():
    x = torch.randn(2, 3, 10, 64, device=DEV, dtype=BF)
    y, mean, rstd = kda.layer_norm_fwd(x)
    y2, none, none2 = kda.layer_norm_fwd(x, want_stats=False)
    assert none is None and none2 is None and torch.equal(y, y2)
    dy = torch.randn_like(x)
    dx, dw, db = kda.layer_norm_bwd(x, None, mean, rstd, dy)
    ws = torch.full((kda.layer_norm_bwd_workspace_bytes(2, 3, 10, 64),), 255, dtype=torch.uint8, device=DEV)
    again = kda.layer_norm_bwd(x, None, mean, rstd, dy, workspace=ws)
    assert all(torch.equal(a, b) for a, b in zip((dx, dw, db), again))
    inplace = dy.clone()
    got, n1, n2 = kda.layer_norm_bwd(x, None, mean, rstd, inplace, want_params=False, dx_out=inplace)
    assert got is inplace and n1 is None and n2 is None and torch.equal(got, dx)
    e = torch.empty(2, 3, 0, 64, device=DEV)
    st = torch.empty(2, 3, 0, device=DEV)
    assert kda.layer_norm_fwd(e)[0].shape == e.shape
    _, dw, db = kda.layer_norm_bwd(e, None, st, st, e)
    torch.cuda.synchronize()
    assert torch.all(dw == 0) and torch.all(db == 0)


def test_long_offsets():
    """Tensors of more than 2^31 elements: the last rows give what they give alone."""
    B, H, T, D = 2, 2, 4300000, 128
    x = torch.zeros((B, H, T, D), dtype=BF, device=DEV)
    assert x.numel() > 2 ** 31
    dy = torch.zeros_like(x)
    x[-1, -1, -500:].normal_()
    dy[-1, -1, -500:].normal_()
    w, b = torch.randn(2, H, D, device=DEV).unbind(0)
    y, mean, rstd = kda.layer_norm_fwd(x, w, b)
    dx, dw, db = kda.layer_norm_bwd(x, w, mean, rstd, dy)
    last = lambda t: t[-1:, -1:, -500:].contiguous()
    y1, m1, r1 = kda.layer_norm_fwd(last(x), w[-1:], b[-1:])
    dx1, dw1, db1 = kda.layer_norm_bwd(last(x), w[-1:], m1, r1, last(dy))
    assert torch.equal(last(y), y1) and torch.equal(last(dx), dx1) and torch.equal(last(mean), m1)
    assert torch.equal(last(rstd), r1)
    # the other rows of the head add zeros to its sums, in another order
    assert norm2(host(dw[-1]), host(dw1[0])) <= F32 and norm2(host(db[-1]), host(db1[0])) <= F32
    assert torch.all(dw[0] == 0) and torch.all(db[0] == 0) and torch.all(y[0, 0, 0] == b[0].to(BF))
