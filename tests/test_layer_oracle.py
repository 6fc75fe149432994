"""The float64 definitions of oracle/layer_ref.py: closed forms, finite differences, and the 8-bit form
against torch's own e4m3 type."""
import numpy as np
import pytest
import torch

from oracle import layer_ref as R


def _attn(rng, B, H, T, K, V):
    n = rng.standard_normal
    return n((B, H, T, K)), n((B, H, T, K)), n((B, H, T, V)), -rng.uniform(0.01, 1.0, H), n((B, H, K, V))


def test_decay_attn_is_the_sum_over_the_past():
    rng = np.random.default_rng(1)
    q, k, v, g, S0 = _attn(rng, 2, 3, 7, 4, 5)
    o, S = R.decay_attn(q, k, v, g, S0, lengths=[7, 4])
    for b, h, t in ((0, 0, 6), (0, 2, 3), (1, 1, 3)):
        want = np.exp(g[h] * (t + 1)) * q[b, h, t] @ S0[b, h]
        for s in range(t + 1):
            want = want + np.exp(g[h] * (t - s)) * (q[b, h, t] @ k[b, h, s]) * v[b, h, s]
        assert np.allclose(o[b, h, t], want * 0.5, rtol=1e-12, atol=1e-12)
    assert np.all(o[1, :, 4:] == 0)
    assert np.allclose(S[1], R.decay_attn(q[1:, :, :4], k[1:, :, :4], v[1:, :, :4], g, S0[1:])[1][0], rtol=1e-13)


def test_decay_attn_limits_of_the_decay():
    rng = np.random.default_rng(2)
    q, k, v, _, S0 = _attn(rng, 1, 2, 5, 4, 4)
    with np.errstate(over="ignore"):
        o, S = R.decay_attn(q, k, v, np.array([-np.inf, 0.0]), S0)
    assert np.allclose(S[0, 0], np.outer(k[0, 0, -1], v[0, 0, -1]))
    assert np.allclose(S[0, 1], S0[0, 1] + k[0, 1].T @ v[0, 1])


def _differences(f, x, h=1e-5):
    g = np.zeros_like(x)
    for i in np.ndindex(*x.shape):
        y = x.copy()
        y[i] += h
        up = f(y)
        y[i] -= 2 * h
        g[i] = (up - f(y)) / (2 * h)
    return g


@pytest.mark.parametrize("lengths", [None, [3, 0]])
def test_decay_attn_adjoint_against_differences(lengths):
    rng = np.random.default_rng(3)
    q, k, v, g, S0 = _attn(rng, 2, 2, 4, 3, 2)
    d_o, dS = rng.standard_normal((2, 2, 4, 2)), rng.standard_normal(S0.shape)
    got = R.decay_attn_adjoint(q, k, v, g, S0, d_o, dS, lengths)

    def loss(q=q, k=k, v=v, S0=S0):
        o, S = R.decay_attn(q, k, v, g, S0, lengths)
        return (o * d_o).sum() + (S * dS).sum()

    for name, x in (("dq", q), ("dk", k), ("dv", v), ("dstate_in", S0)):
        arg = {"dq": "q", "dk": "k", "dv": "v", "dstate_in": "S0"}[name]
        ref = _differences(lambda y: loss(**{arg: y}), x)
        assert np.abs(got[name] - ref).max() <= 1e-8 * max(1.0, np.abs(ref).max()), name


def test_layer_norm_adjoint_against_differences():
    rng = np.random.default_rng(4)
    x, w, b = rng.standard_normal((2, 2, 3, 5)), rng.standard_normal((2, 5)), rng.standard_normal((2, 5))
    dy = rng.standard_normal(x.shape)
    _, mean, rstd = R.layer_norm(x, w, b)
    dx, dw, db = R.layer_norm_adjoint(x, w, mean, rstd, dy)
    f = lambda x=x, w=w, b=b: (R.layer_norm(x, w, b)[0] * dy).sum()
    assert np.abs(dx - _differences(lambda y: f(x=y), x)).max() <= 1e-8
    assert np.abs(dw - _differences(lambda y: f(w=y), w)).max() <= 1e-8
    assert np.abs(db - _differences(lambda y: f(b=y), b)).max() <= 1e-8


def test_ckpt_codes_are_torchs_e4m3():
    rng = np.random.default_rng(5)
    for D in (8, 24, 64):
        x = (rng.standard_normal((50, D)) * 2.0 ** rng.integers(-30, 30, (50, 1))).astype(np.float32)
        x[0] = 0.0
        x[1, :3] = (448.0, -448.0, 0.5)
        codes, scales = R.ckpt_pack(x)
        G = min(D, 32)
        y = torch.from_numpy(x).double().reshape(50, D // G, G)
        y = y * torch.exp2(127.0 - torch.from_numpy(scales.astype(np.float64))).unsqueeze(-1)
        want = y.float().to(torch.float8_e4m3fn).view(torch.uint8).reshape(50, D)
        assert torch.equal(torch.from_numpy(codes), want)
        back = R.ckpt_unpack(codes, scales)
        # nearest value: half a step of e4m3 (2^-4 relative), or of its subnormals (2^-10 of the scale)
        s = np.repeat(2.0 ** (scales.astype(np.float64) - 127), G, -1)
        assert np.all(np.abs(back - x) <= np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -10 * s))
    codes, scales = R.ckpt_pack(np.array([[np.inf, -np.inf, np.nan, 1.0] + [0.0] * 4]))
    assert np.all(np.isnan(R.ckpt_unpack(codes, scales)[0, :3])) and R.ckpt_unpack(codes, scales)[0, 3] == 1.0
