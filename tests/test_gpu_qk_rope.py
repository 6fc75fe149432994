"""Norm of queries and keys with the rotation by position on the GPU against float64.

Tolerances, element by element, with e = 2^-24, U = 2^-8 for a rounding to bf16 (fp32: e):
  r           a sum of D <= 256 squares in 8 + 5 additions, a product, a sum, a reciprocal root: 12 e of itself
  cos, sin    the part of a turn rounded to fp32 (2^-25 of at most 1/2, times 2 pi: 1.6 e) and the function (2 e), the scale (e)
  y           the products x (r w), both rounded, times cos or sin, two of them added: (12 + 3 + 5 + 3) e (|u| + |v|) scale
              for a pair, at most 24 e
  dx          p = Rot^T dy (8 e), p w (9 e), xh (13 e), their dot product (9 + 13 + 15 e of the absolute sum), the
              difference and the product with r: 60 e r (|p w| + |xh| mean |p w xh|)
  dw          a sum over rows: 21 e of each term, N additions one behind the other: 64 rows of a lane (32 blocks of 2 heads' worth at
              most 8 heads: 256), 256 / L lanes, a sixteenth of the parts and 16
"""
import numpy as np
import pytest
import torch

import gated_delta_rule_47_amd as kda
from oracle import sequence_ref as R

from gpu_helpers import DEV, host, say, to_dev

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float32
E32 = 2.0 ** -24
U = {BF: 2.0 ** -8, FP: E32}


def within(name, got, ref, lim):
    g = host(got)
    assert g.shape == ref.shape, name
    over = np.abs(g - ref) - lim
    assert np.all(over <= 0), (name, float(over.max()), np.unravel_index(over.argmax(), over.shape))


def _pairs(a, n, inter):
    """Of every channel, the sum of its pair's absolute values (its own alone where it is not rotated)."""
    out = a.copy()
    i = np.arange(0, 2 * n, 2) if inter else np.arange(n)
    j = i + 1 if inter else i + n
    out[..., i] = out[..., j] = a[..., i] + a[..., j]
    return out


def _opt(t):
    return None if t is None else host(t)


def check(B, T, Hq, Hk, D, R_, dtype, norm="rms", rows=(1, 1), inter=False, positions=None, scale=1.0, eps=1e-6, seed=0):
    say("qk", B, T, Hq, Hk, D, R_, dtype, norm, rows, inter)
    rng = np.random.default_rng(seed)
    n = (Hq + Hk + 1) * D
    fused = to_dev(rng.standard_normal((B, T, n)) * np.exp(rng.standard_normal((1, 1, n))), dtype)
    q = fused[..., :Hq * D].view(B, T, Hq, D)
    k = fused[..., Hq * D:(Hq + Hk) * D].view(B, T, Hk, D) if Hk else None
    w = [None if norm is None or r == 0 else to_dev(1 + 0.3 * rng.standard_normal((r, D)), FP) for r in rows]
    f = None if R_ == 0 else kda.rope_frequencies(R_, device=DEV)[0]
    pos = None if positions is None else torch.tensor(positions, dtype=torch.int32, device=DEV)
    how = dict(positions=pos, norm=norm, q_weight=w[0], k_weight=w[1] if Hk else None, eps=eps, interleaved=inter, rope_scale=scale)
    yq, yk = kda.qk_norm_rope_fwd(q, k, f, **how)
    torch.cuda.synchronize()
    dq, dk = to_dev(rng.standard_normal((B, Hq, T, D)), dtype), to_dev(rng.standard_normal((B, Hk, T, D)), dtype) if Hk else None
    grad = torch.full_like(fused, 5.0)
    oq = grad[..., :Hq * D].view(B, T, Hq, D)
    ok = grad[..., Hq * D:(Hq + Hk) * D].view(B, T, Hk, D) if Hk else None
    g = kda.qk_norm_rope_bwd(q, k, f, dq, dk, dq_out=oq, dk_out=ok, **how)
    torch.cuda.synchronize()
    assert torch.all(grad[..., (Hq + Hk) * D:] == 5)
    if not Hk:
        assert yk is None and g["dk"] is None and g["dk_weight"] is None
    fr = np.zeros(0) if f is None else host64(f)
    nr = R_ // 2
    for x, y, dy, dx, ww, dw in ((q, yq, dq, g["dq"], w[0], g["dq_weight"]), (k, yk, dk, g["dk"], w[1], g["dk_weight"])):
        if x is None:
            continue
        xx, wn = host(x), _opt(ww)
        ref = R.qk_norm_rope(xx, wn, fr, positions, norm, eps, inter, scale)
        r = R._qk_rows(xx, norm, eps)
        xn = np.abs(xx * r * (1 if wn is None else wn))
        mag = _pairs(xn, nr, inter).transpose(0, 2, 1, 3) * max(1.0, abs(scale))
        within("y", y, ref, 24 * E32 * mag + U[dtype] * np.abs(ref))
        rdx, rdw = R.qk_norm_rope_adjoint(xx, wn, fr, host(dy), positions, norm, eps, inter, scale)
        p = _pairs(np.abs(host(dy)).transpose(0, 2, 1, 3), nr, inter) * max(1.0, abs(scale))
        pw, xh = p * (1 if wn is None else np.abs(wn)), np.abs(xx * r)
        m = r * pw
        if norm is not None:
            m = r * (pw + xh * ((pw * xh).mean(-1, keepdims=True) if norm == "rms" else (pw * xh).sum(-1, keepdims=True)))
        within("dx", dx, rdx, 60 * E32 * m + U[dtype] * np.abs(rdx))
        if ww is None:
            assert dw is None
            continue
        per = p * xh
        per = per.sum((0, 1)) if ww.shape[0] > 1 else per.sum((0, 1, 2))[None]
        N = 256 + 256 + B * T * (Hq + Hk) / 16 + 16
        within("dw", dw, rdw, (21 + min(N, B * T * (1 if ww.shape[0] > 1 else Hq + Hk))) * E32 * per)
    return yq, yk


def host64(t):
    return t.detach().cpu().numpy()


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("D", [8, 16, 24, 32, 40, 64, 80, 96, 128, 136, 192, 256])
def test_head_widths(D, dtype):
    check(2, 5, 3, 2, D, D, dtype, seed=D)
    check(1, 7, 2, 2, D, D // 16 * 8, dtype, "l2", inter=True, seed=D)
    check(1, 3, 1, 1, D, 8, dtype, None, seed=D)


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("R_", [0, 8, 16, 56, 64])
def test_rotated_parts(R_, inter, dtype):
    check(2, 9, 2, 1, 64, R_, dtype, inter=inter, seed=R_)
    check(2, 9, 2, 1, 64, R_, dtype, None, inter=inter, scale=1.25, seed=R_)


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("B,T,Hq,Hk", [(1, 1, 1, 1), (1, 1, 32, 8), (200, 1, 4, 4), (3, 257, 8, 2), (1, 1000, 5, 0), (2, 63, 1, 9),
                                       (7, 65, 33, 31)])
def test_tokens_and_heads(B, T, Hq, Hk, dtype):
    check(B, T, Hq, Hk, 32, 32, dtype, seed=T)


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("rows", [(4, 1), (1, 2), (4, 2), (0, 2), (4, 0), (0, 0)])
@pytest.mark.parametrize("norm", ["rms", "l2"])
def test_weights_per_head_or_shared(rows, norm, dtype):
    check(2, 50, 4, 2, 40, 24, dtype, norm, rows, seed=rows[0])


def test_more_workgroups_and_several_blocks_of_tokens():
    check(2, 9000, 8, 8, 64, 64, BF, seed=3)
    check(1, 12000, 4, 4, 128, 128, FP, "l2", (4, 4), seed=4)


def test_far_positions():
    """Angles of 2^31 radians and their neighbours, which a float32 would hold to 128 radians.  In float64 the position times the
    frequency, times 1 / (2 pi) as a constant, is off by 3 2^-53 of itself: 6 in units of 2^-24 radians at 2^31, beside the
    8 of an angle and its function; without a norm 16 of the 24 are free for them."""
    pos = [[0, 1, 2, -1, -2 ** 31, 2 ** 31 - 1, 10 ** 6, 10 ** 9, -10 ** 9, 123456789]]
    check(1, 10, 2, 2, 64, 64, FP, None, positions=pos, seed=7)


def test_scaled_frequencies():
    """Scaled tables go through the same kernel: the rotation by parts against the definition."""
    B, T, H, D = 1, 40, 2, 64
    rng = np.random.default_rng(5)
    x = to_dev(rng.standard_normal((B, T, H, D)), FP)
    pos = np.arange(T)[None] * 997
    for scaling, kw in (("linear", dict(factor=4.0)), ("base", dict(factor=4.0)), ("parts", dict(factor=16.0))):
        f, s = kda.rope_frequencies(D, scaling=scaling, device=DEV, **kw)
        rf, rs = R.rope_frequencies(D, scaling=scaling, **kw)
        y, _ = kda.qk_norm_rope_fwd(x, None, f, to_dev(pos, torch.int32), norm=None, rope_scale=s)
        ref = R.qk_norm_rope(host(x), None, rf, pos, None, rope_scale=rs)
        mag = _pairs(np.abs(host(x)), D // 2, False).transpose(0, 2, 1, 3) * rs
        within(scaling, y, ref, 24 * E32 * mag)


@pytest.mark.parametrize("dtype", [BF, FP])
def test_any_strides(dtype):
    """Heads outermost, batch inside the token, a broadcast batch, rows off any alignment."""
    B, T, H, D = 2, 21, 3, 32
    rng = np.random.default_rng(6)
    x = to_dev(rng.standard_normal((B, T, H, D)), dtype)
    f = kda.rope_frequencies(D, device=DEV)[0]
    w = to_dev(1 + 0.1 * rng.standard_normal((1, D)), FP)
    dy = to_dev(rng.standard_normal((B, H, T, D)), dtype)
    want, _ = kda.qk_norm_rope_fwd(x, None, f, q_weight=w)
    ref = kda.qk_norm_rope_bwd(x, None, f, dy, None, q_weight=w)
    for order in ((2, 0, 1), (1, 0, 2), (0, 2, 1), (1, 2, 0)):
        back = [order.index(i) for i in range(3)] + [3]
        shape = [x.shape[i] for i in order]
        buf = torch.zeros(shape + [D + 5], dtype=dtype, device=DEV)
        v = buf[..., 3:3 + D].permute(back)
        v.copy_(x)
        got, _ = kda.qk_norm_rope_fwd(v, None, f, q_weight=w)
        assert torch.equal(got, want), order
        out = torch.full_like(buf, 5.0)
        o = out[..., 3:3 + D].permute(back)
        g = kda.qk_norm_rope_bwd(v, None, f, dy, None, q_weight=w, dq_out=o)
        assert torch.equal(o, ref["dq"]) and torch.equal(g["dq_weight"], ref["dq_weight"])
        o.fill_(5.0)
        assert torch.all(out == 5)
    one = x[:1].expand(B, T, H, D)
    got, _ = kda.qk_norm_rope_fwd(one, None, f, q_weight=w)
    assert torch.equal(got[1], want[0]) and torch.equal(got[0], want[0])


def test_keys_beside_queries_and_alone_agree():
    B, T, D = 2, 30, 64
    q, k = torch.randn(B, T, 4, D, device=DEV).to(BF), torch.randn(B, T, 2, D, device=DEV).to(BF)
    f = kda.rope_frequencies(D, device=DEV)[0]
    yq, yk = kda.qk_norm_rope_fwd(q, k, f)
    assert torch.equal(yq, kda.qk_norm_rope_fwd(q, None, f)[0]) and torch.equal(yk, kda.qk_norm_rope_fwd(k, None, f)[0])
    same, _ = kda.qk_norm_rope_fwd(q, q, f)                        # one tensor for both
    assert torch.equal(same, yq)


def test_tokens_one_by_one_continue_a_prompt():
    B, T, H, D = 3, 17, 4, 64
    q, k = torch.randn(B, T, H, D, device=DEV).to(BF), torch.randn(B, T, H, D, device=DEV).to(BF)
    f = kda.rope_frequencies(D, device=DEV)[0]
    pos = (torch.tensor([[5], [70000], [0]], device=DEV) + torch.arange(T, device=DEV)).to(torch.int32)
    yq, yk = kda.qk_norm_rope_fwd(q, k, f, pos, norm="l2")
    for t in (0, 9, 16):
        aq, ak = kda.qk_norm_rope_fwd(q[:, t:t + 1], k[:, t:t + 1], f, pos[:, t:t + 1].contiguous(), norm="l2")
        assert torch.equal(aq[:, :, 0], yq[:, :, t]) and torch.equal(ak[:, :, 0], yk[:, :, t])


def test_zero_and_non_finite_rows():
    f = kda.rope_frequencies(32, device=DEV)[0]
    x = torch.randn(1, 6, 2, 32, device=DEV)
    x[0, 1, 0] = 0
    x[0, 2, 1, 5] = float("nan")
    x[0, 3, 0, 7] = float("inf")
    w = torch.ones(1, 32, device=DEV)
    y, _ = kda.qk_norm_rope_fwd(x, None, f, q_weight=w)
    assert torch.all(y[0, 0, 1] == 0) and torch.isnan(y[0, 1, 2]).all() and torch.isnan(y[0, 0, 3]).any()
    fine = torch.ones(2, 6, dtype=torch.bool, device=DEV)
    fine[1, 2] = fine[0, 3] = False
    assert torch.isfinite(y[0][fine]).all()                        # rows keep to themselves
    y, _ = kda.qk_norm_rope_fwd(x, None, f, eps=0.0)
    assert torch.isnan(y[0, 0, 1]).all()                           # 0 / 0, as the formula
    z = torch.zeros(1, 3, 2, 32, device=DEV)                       # partial workgroups' idle lanes add nothing
    z[..., 0] = 1
    g = kda.qk_norm_rope_bwd(z, None, f, torch.ones(1, 2, 3, 32, device=DEV), None, q_weight=w, eps=0.0)
    assert torch.isfinite(g["dq_weight"]).all() and torch.isfinite(g["dq"]).all()


def test_gradients_of_weights_that_are_not_given():
    """The C entry takes the weights' gradients without weights (ones), a row per head or one for all, and keys alone."""
    from gated_delta_rule_47_amd import _lib
    lib = _lib.load()
    B, T, H, D = 2, 40, 3, 32
    x, dy = torch.randn(B, T, H, D, device=DEV), torch.randn(B, H, T, D, device=DEV)
    f = kda.rope_frequencies(D, device=DEV)[0]
    st = x.stride()[:3]
    for rows in (1, H):
        want = kda.qk_norm_rope_bwd(x, None, f, dy, None, q_weight=torch.ones(rows, D, device=DEV))
        for keys in (False, True):
            dx, dw = torch.zeros_like(x), torch.zeros(rows, D, device=DEV)
            need = lib.kda_qk_norm_rope_bwd_workspace_bytes(B, T, 0 if keys else H, 1 if keys else rows, H if keys else 0, rows, D)
            ws = torch.empty(need, dtype=torch.uint8, device=DEV)
            side, none = (x.data_ptr(), *st), (None, 0, 0, 0)
            out = (dx.data_ptr(), *st)
            a = (none, side) if keys else (side, none)
            o = (none, out) if keys else (out, none)
            r = lib.kda_qk_norm_rope_bwd(*a[0], *a[1], None, 1 if keys else rows, None, rows, 1, 1e-6, f.data_ptr(), None, 1.0, 0,
                                         None if keys else dy.data_ptr(), dy.data_ptr() if keys else None, *o[0], *o[1],
                                         None if keys else dw.data_ptr(), dw.data_ptr() if keys else None, ws.data_ptr(), need,
                                         B, T, 0 if keys else H, H if keys else 0, D, D, 0, torch.cuda.current_stream().cuda_stream)
            torch.cuda.synchronize()
            assert r == 0 and torch.equal(dx, want["dq"]) and torch.equal(dw, want["dq_weight"]), (rows, keys)


def test_no_tokens():
    x = torch.empty(2, 0, 3, 16, device=DEV)
    f = kda.rope_frequencies(16, device=DEV)[0]
    w = torch.ones(1, 16, device=DEV)
    y, k = kda.qk_norm_rope_fwd(x, x, f, q_weight=w, k_weight=w)
    assert y.shape == (2, 3, 0, 16) and k.shape == (2, 3, 0, 16)
    g = kda.qk_norm_rope_bwd(x, x, f, y, k, q_weight=w, k_weight=w)
    assert not g["dq_weight"].any() and not g["dk_weight"].any()


def test_gradient_against_differences_of_the_kernel():
    """Along random directions: the loss is a float64 sum of 4096 terms of size 1, each off by 24 e or so, over 2 h = 2^-6:
    sqrt(4096) 24 2^-24 2^6 = 6e-3; the cubic term h^2 / 6 of derivatives of size 10 of 4096 terms with either sign, 64 4e-4."""
    B, T, H, D = 2, 16, 2, 64
    rng = np.random.default_rng(9)
    x, dy = to_dev(rng.standard_normal((B, T, H, D)), FP), to_dev(rng.standard_normal((B, H, T, D)), FP)
    w = to_dev(1 + 0.2 * rng.standard_normal((2, D)), FP)
    f = kda.rope_frequencies(32, device=DEV)[0]
    for norm in ("rms", "l2"):
        g = kda.qk_norm_rope_bwd(x, None, f, dy, None, norm=norm, q_weight=w)
        loss = lambda x, w: float((kda.qk_norm_rope_fwd(x, None, f, norm=norm, q_weight=w)[0].double() * dy).sum())
        h = 2.0 ** -7
        v, u = torch.randn_like(x), torch.randn_like(w)
        for fd, an in (((loss(x + h * v, w) - loss(x - h * v, w)) / (2 * h), float((g["dq"].double() * v).sum())),
                       ((loss(x, w + h * u) - loss(x, w - h * u)) / (2 * h), float((g["dq_weight"].double() * u).sum()))):
            assert abs(fd - an) <= 0.03 + 2e-3 * abs(an), (norm, fd, an)


def test_offsets_past_32_bits():
    """A fused projection of more than 2^31 elements: the last tokens give what they give alone."""
    T, Hq, Hk, D = 180000, 64, 16, 128
    x = torch.zeros((1, T, (Hq + 2 * Hk) * D), dtype=BF, device=DEV)
    assert x.numel() > 2 ** 31
    n = 70
    x[:, -n:].normal_()
    f = kda.rope_frequencies(D, device=DEV)[0]
    pos = torch.arange(T, device=DEV, dtype=torch.int32)[None]
    split = lambda t: (t[..., :Hq * D].unflatten(-1, (Hq, D)), t[..., Hq * D:(Hq + Hk) * D].unflatten(-1, (Hk, D)))
    yq, yk = kda.qk_norm_rope_fwd(*split(x), f, pos)
    aq, ak = kda.qk_norm_rope_fwd(*split(x[:, -n:]), f, pos[:, -n:].contiguous())
    assert torch.equal(yq[:, :, -n:], aq) and torch.equal(yk[:, :, -n:], ak)
    grad = torch.zeros_like(x)
    oq, ok = split(grad)
    kda.qk_norm_rope_bwd(*split(x), f, yq, yk, pos, dq_out=oq, dk_out=ok)
    g = kda.qk_norm_rope_bwd(*split(x[:, -n:]), f, aq, ak, pos[:, -n:].contiguous())
    assert torch.equal(oq[:, -n:], g["dq"]) and torch.equal(ok[:, -n:], g["dk"]) and not grad[..., (Hq + Hk) * D:].any()
