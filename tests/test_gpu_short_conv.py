"""Short causal convolution on the GPU against float64.

Tolerances, element by element: one rounding to bf16 is off by at most U = 2^-8 of the value (fp32: 2^-24), and the fp32
arithmetic before it, with e = 2^-24, M = |bias| + sum |w x|:
  pre          (W + 1) e M
  y = pre s    its derivative is at most 1.1, s (an exponential, a sum, a reciprocal, the argument's rounding) off by
               (|pre| + 8) e of itself: 1.1 (W + 1) e M + (|pre| + 8) e |y|
  dpre         dy (s + pre s (1 - s)), whose derivative is at most 0.5: |dy| (0.6 (W + 1) e M + 1.1 (|pre| + 10) e) + 4 e |dpre|
  dx, dstate   sums of W products of w and dpre: those errors through |w|, and (W + 2) e of the absolute sum
  dw, db       those errors through |x|, and N e of the absolute sum for N additions one behind the other: at most 128 tokens
               of a run, 256 runs of a workgroup, a sixteenth of the parts and 16
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


def inputs(B, T, C, W, dtype, seed, bias=True, state=True):
    rng = np.random.default_rng(seed)
    n = rng.standard_normal
    x, w = to_dev(n((B, T, C)), dtype), to_dev(n((C, W)) * W ** -0.5, FP)
    return x, w, to_dev(n(C), FP) if bias else None, to_dev(n((B, W - 1, C)), dtype) if state else None


def _opt(t):
    return None if t is None else host(t)


def limits(x, w, b, s, dy, lengths, silu, heads):
    """(limit of y (B,H,T,D) before its rounding, of dpre (B,T,C), |dpre|)."""
    B, T, C = x.shape
    W = w.shape[-1]
    xx, ww, ss = host(x), host(w), _opt(s)
    full, pre = R._conv_pre(xx, ww, _opt(b), ss)
    M = R._conv_pre(np.abs(xx), np.abs(ww), None if b is None else np.abs(host(b)), None if ss is None else np.abs(ss))[1]
    y = pre / (1 + np.exp(-pre)) if silu else pre
    ly = (1.1 * (W + 1) * E32 * M + (np.abs(pre) + 8) * E32 * np.abs(y)) if silu else (W + 1) * E32 * M
    ly = ly.reshape(B, T, heads, C // heads).transpose(0, 2, 1, 3)
    if dy is None:
        return ly, None, None, full
    d = np.abs(host(dy)).transpose(0, 2, 1, 3).reshape(B, T, C)
    g = 1 / (1 + np.exp(-pre))
    dp = d * np.abs(g + pre * g * (1 - g)) if silu else d
    ld = d * (0.6 * (W + 1) * E32 * M + 1.1 * (np.abs(pre) + 10) * E32) + 4 * E32 * dp if silu else 0 * d
    for bb, n in enumerate(R._lens(lengths, B, T)):
        dp[bb, n:] = ld[bb, n:] = 0
    return ly, ld, dp, full


def check(B, T, H, D, W, dtype, lengths=None, silu=True, bias=True, state=True, seed=0, x=None, backward=True):
    C = H * D
    say("conv", B, T, H, D, W, dtype, lengths, silu, bias, state)
    x0, w, b, s = inputs(B, T, C, W, dtype, seed, bias, state)
    x = x0 if x is None else x(x0)
    lens = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device=DEV)
    act = "silu" if silu else None
    out = torch.full((B, H, T, D), 7.0, dtype=dtype, device=DEV)
    y, end = kda.short_conv_fwd(x, w, b, s, lengths=lens, activation=act, heads=H, out=out)
    torch.cuda.synchronize()
    dy = to_dev(np.random.default_rng(seed + 1).standard_normal((B, H, T, D)), dtype)
    ry, rend = R.short_conv(host(x), host(w), _opt(b), _opt(s), lengths, silu, H)
    ly, ld, dp, full = limits(x, w, b, s, dy, lengths, silu, H)
    for bb, n in enumerate(R._lens(lengths, B, T)):
        assert torch.all(out[bb, :, n:] == 7)              # rows behind a sequence stay
        ry[bb, :, n:] = 7
    within("y", y, ry, ly + U[dtype] * np.abs(ry))
    assert np.array_equal(host(end), rend)                 # inputs, copied
    if not backward:
        return
    ds = to_dev(np.random.default_rng(seed + 2).standard_normal((B, W - 1, C)), FP)
    got = kda.short_conv_bwd(x, w, b, s, dy, ds, lens, act)
    torch.cuda.synchronize()
    ref = R.short_conv_adjoint(host(x), host(w), _opt(b), _opt(s), host(dy), host(ds), lengths, silu)
    aw = np.abs(host(w))
    lfull, afull = np.zeros_like(full), np.zeros_like(full)
    ldw, adw = np.zeros_like(aw), np.zeros_like(aw)
    for j in range(W):
        lfull[:, j:j + T] += aw[:, j] * ld
        afull[:, j:j + T] += aw[:, j] * dp
        ldw[:, j] = (np.abs(full[:, j:j + T]) * ld).sum((0, 1))
        adw[:, j] = (np.abs(full[:, j:j + T]) * dp).sum((0, 1))
    for bb, n in enumerate(R._lens(lengths, B, T)):
        afull[bb, n:n + W - 1] += np.abs(host(ds)[bb])
    lim = lfull + (W + 2) * E32 * afull
    within("dx", got["dx"], ref["dx"], lim[:, W - 1:] + U[dtype] * np.abs(ref["dx"]))
    within("dstate_in", got["dstate_in"], ref["dstate_in"], lim[:, :W - 1] + E32 * np.abs(ref["dstate_in"]))
    N = 128 + 256 + B * (T // 8 + 1) / 16 + 16
    within("dweight", got["dweight"], ref["dweight"], ldw + N * E32 * adw)
    within("dbias", got["dbias"], ref["dbias"], ld.sum((0, 1)) + N * E32 * dp.sum((0, 1)))
    return got


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("T", [1, 2, 3, 4, 7, 8, 9, 33, 257])
def test_lengths_and_widths(T, W, dtype):
    check(2, T, 2, 8, W, dtype, seed=T)
    check(1, T, 1, 24, W, dtype, silu=False, bias=False, state=False, seed=T + 1)


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("H,D", [(1, 8), (1, 16), (3, 8), (5, 40), (1, 520), (4, 128), (96, 8), (1, 4104)])
def test_channels(H, D, dtype):
    check(2, 40, H, D, 4, dtype, seed=H * D)


@pytest.mark.parametrize("dtype", [BF, FP])
def test_padded_batches(dtype):
    check(6, 50, 2, 32, 4, dtype, lengths=[50, 0, 1, 2, 49, 17])
    check(3, 50, 2, 32, 3, dtype, lengths=[-5, 99, 8], silu=False)
    check(2, 3, 1, 8, 4, dtype, lengths=[1, 2], state=False)


def test_long_sequences_and_runs():
    check(3, 5000, 4, 64, 4, BF, lengths=[5000, 4097, 128])       # runs of more than eight tokens
    check(1, 20011, 2, 128, 4, FP)
    check(33, 70, 8, 64, 4, BF)


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("shift", [0, 1, 3])
def test_slices_of_a_wider_projection(dtype, shift):
    """x and dx between the rows of wider tensors, off any alignment, the batch inside the token's stride too."""
    B, T, C, W = 2, 37, 48, 4
    wide = C + 19
    x, w, b, s = inputs(B, T, C, W, dtype, 3)
    dy = to_dev(np.random.default_rng(4).standard_normal((B, 3, T, 16)), dtype)
    want = kda.short_conv_fwd(x, w, b, s, heads=3)
    ref = kda.short_conv_bwd(x, w, b, s, dy)
    for time_first in (False, True):
        buf = torch.full((T, B, wide) if time_first else (B, T, wide), 5.0, dtype=dtype, device=DEV)
        view = (buf.transpose(0, 1) if time_first else buf)[..., shift:shift + C]
        view.copy_(x)
        got = kda.short_conv_fwd(view, w, b, s, heads=3)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        gbuf = torch.full_like(buf, 5.0)
        gview = (gbuf.transpose(0, 1) if time_first else gbuf)[..., shift:shift + C]
        r = kda.short_conv_bwd(view, w, b, s, dy, dx_out=gview)
        assert r["dx"] is gview and torch.equal(gview, ref["dx"]) and torch.equal(r["dweight"], ref["dweight"])
        gview.fill_(5.0)
        assert torch.all(gbuf == 5)                                # nothing beside it was touched
    step = kda.short_conv_step(buf.view(-1, wide)[:4, shift:shift + C], w, b, torch.zeros(4, 3, C, dtype=dtype, device=DEV))
    assert step.shape == (4, C)


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("W", [2, 3, 4])
def test_steps_continue_a_prompt(W, dtype):
    """Token by token gives what the whole sequence gives, bit by bit."""
    B, T, H, D = 3, 12, 2, 16
    x, w, b, s = inputs(B, T, H * D, W, dtype, 9)
    y, end = kda.short_conv_fwd(x, w, b, s, heads=H)
    y1, state = kda.short_conv_fwd(x[:, :5], w, b, s, heads=H)
    assert torch.equal(y1, y[:, :, :5])
    for t in range(5, T):
        yt = kda.short_conv_step(x[:, t], w, b, state)
        assert torch.equal(yt.view(B, H, D), y[:, :, t]), t
    assert torch.equal(state, end)


def test_no_tokens():
    x, w, b, s = inputs(2, 0, 16, 4, BF, 1)
    y, end = kda.short_conv_fwd(x, w, b, s)
    assert y.shape == (2, 1, 0, 16) and torch.equal(end, s)
    _, end = kda.short_conv_fwd(x, w, b, None)
    assert not end.any()
    ds = torch.randn(2, 3, 16, device=DEV)
    r = kda.short_conv_bwd(x, w, b, s, y, ds)
    assert torch.equal(r["dstate_in"], ds) and not r["dweight"].any() and not r["dbias"].any()
    r = kda.short_conv_bwd(x, w, b, s, y, want_params=False)
    assert not r["dstate_in"].any() and r["dweight"] is None


def test_non_finite_values_keep_to_what_reads_them():
    B, T, H, D, W = 2, 30, 1, 16, 4
    x, w, b, s = inputs(B, T, H * D, W, FP, 5)
    lens = torch.tensor([30, 10], dtype=torch.int32, device=DEV)
    y0, e0 = kda.short_conv_fwd(x, w, b, s, lengths=lens, out=torch.zeros(B, H, T, D, device=DEV))
    dy = torch.randn(B, H, T, D, device=DEV)
    g0 = kda.short_conv_bwd(x, w, b, s, dy, lengths=lens)
    bad, dbad = x.clone(), dy.clone()
    bad[1, 10:] = float("nan")                                     # behind the sequence: never read
    dbad[1, :, 10:] = float("inf")
    y1, e1 = kda.short_conv_fwd(bad, w, b, s, lengths=lens, out=torch.zeros(B, H, T, D, device=DEV))
    g1 = kda.short_conv_bwd(bad, w, b, s, dbad, lengths=lens)
    assert torch.equal(y0, y1) and torch.equal(e0, e1) and all(torch.equal(g0[k], g1[k]) for k in g0)
    bad = x.clone()
    bad[0, 4, 3] = float("inf")
    y2, _ = kda.short_conv_fwd(bad, w, b, s)
    hit = ~torch.isfinite(y2) | (y2 != kda.short_conv_fwd(x, w, b, s)[0])
    assert not hit[1].any() and not hit[0, 0, :4].any() and not hit[0, 0, 8:].any() and not hit[0, 0, :, :3].any()


def test_gradients_against_differences_of_the_kernel():
    """Central differences of the fp32 forward itself along random directions: the loss is a sum of about 2000 terms of size
    1 in float64, each output off by 2^-24 |y| or so, so a difference over 2 h = 2^-5 is off by sqrt(2000) 2^-24 2^5 = 9e-5, and
    the cubic term by h^2 / 6 of third derivatives of size 10: 4e-4 of |v|^3 terms; the directional derivative is of size 40."""
    B, T, H, D, W = 2, 16, 2, 32, 4
    x, w, b, s = inputs(B, T, H * D, W, FP, 21)
    dy = torch.randn(B, H, T, D, device=DEV)
    ds = torch.randn(B, W - 1, H * D, device=DEV)
    g = kda.short_conv_bwd(x, w, b, s, dy, ds)

    def loss(x, w, b, s):
        y, e = kda.short_conv_fwd(x, w, b, s, heads=H)
        return float((y.double() * dy).sum() + (e.double() * ds).sum())

    h = 2.0 ** -6
    for k, name in enumerate(("dx", "dweight", "dbias", "dstate_in")):
        args = [x, w, b, s]
        v = torch.randn_like(args[k]) * 0.3
        up, dn = list(args), list(args)
        up[k], dn[k] = args[k] + h * v, args[k] - h * v
        fd = (loss(*up) - loss(*dn)) / (2 * h)
        an = float((g[name].double() * v).sum())
        assert abs(fd - an) <= 1e-2 + 2e-3 * abs(an), (name, fd, an)


def test_offsets_past_32_bits():
    """More than 2^32 bytes and 2^31 elements: the last tokens give what they give alone."""
    B, T, C, W = 2, 140000, 8192, 4
    x = torch.zeros((B, T, C), dtype=BF, device=DEV)
    assert x.numel() > 2 ** 31
    n = 200
    x[-1, -n:].normal_()
    _, w, b, _ = inputs(1, 1, C, W, BF, 2)
    y, end = kda.short_conv_fwd(x, w, b, heads=64)
    tail = torch.zeros((1, n + 8, C), dtype=BF, device=DEV)
    tail[:, 8:] = x[-1:, -n:]
    y1, end1 = kda.short_conv_fwd(tail, w, b, heads=64)
    assert torch.equal(y[-1:, :, -n:], y1[:, :, 8:]) and torch.equal(end[-1:], end1)
    dy = y.zero_()
    dy[-1, :, -n:] = torch.randn(64, n, C // 64, device=DEV).to(BF)
    d1 = torch.zeros_like(y1)
    d1[:, :, 8:] = dy[-1:, :, -n:]
    r, r1 = kda.short_conv_bwd(x, w, b, None, dy), kda.short_conv_bwd(tail, w, b, None, d1)
    assert torch.equal(r["dx"][-1:, -n:], r1["dx"][:, 8:])
    assert (host(r["dweight"]) - host(r1["dweight"])).__abs__().max() <= 600 * E32 * n * 20
    assert not r["dx"][0].any()
