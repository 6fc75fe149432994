"""The float64 definitions of oracle/sequence_ref.py: closed forms, invariants and finite differences."""
import numpy as np
import pytest

from oracle import sequence_ref as R


def _differences(f, x, h=1e-5):
    g = np.zeros_like(x)
    for i in np.ndindex(*x.shape):
        y = x.copy()
        y[i] += h
        up = f(y)
        y[i] -= 2 * h
        g[i] = (up - f(y)) / (2 * h)
    return g


def _close(a, b, tol=1e-8):
    assert np.abs(a - b).max(initial=0.0) <= tol * max(1.0, np.abs(b).max(initial=0.0))


# ------------------------------------------------------------------ short convolution
def test_conv_is_a_convolution_and_splits_anywhere():
    rng = np.random.default_rng(1)
    x, w, b, s = rng.standard_normal((2, 9, 6)), rng.standard_normal((6, 4)), rng.standard_normal(6), rng.standard_normal((2, 3, 6))
    y, end = R.short_conv(x, w, b, s, silu=False, heads=3)
    full = np.concatenate((s, x), 1)
    for bb, c in ((0, 0), (1, 5)):
        want = np.convolve(full[bb, :, c], w[c, ::-1], "valid") + b[c]
        assert np.allclose(y[bb, c // 2, :, c % 2], want, atol=1e-12)
    assert np.array_equal(end, full[:, -3:])
    y1, mid = R.short_conv(x[:, :2], w, b, s, silu=False, heads=3)
    y2, end2 = R.short_conv(x[:, 2:], w, b, mid, silu=False, heads=3)
    assert np.allclose(np.concatenate((y1, y2), 2), y) and np.array_equal(end2, end)
    short = R.short_conv(x, w, b, s, lengths=[1, 0])[1]
    assert np.array_equal(short[0], full[0, 1:4]) and np.array_equal(short[1], s[1])


@pytest.mark.parametrize("silu", [True, False])
@pytest.mark.parametrize("lengths", [None, [4, 0, 1]])
def test_conv_adjoint_against_differences(silu, lengths):
    rng = np.random.default_rng(2)
    B, T, C, W = 3, 4, 4, 3
    x, w, b = rng.standard_normal((B, T, C)), rng.standard_normal((C, W)), rng.standard_normal(C)
    s, dy, ds = rng.standard_normal((B, W - 1, C)), rng.standard_normal((B, 2, T, C // 2)), rng.standard_normal((B, W - 1, C))

    def loss(x=x, w=w, b=b, s=s):
        y, e = R.short_conv(x, w, b, s, lengths, silu, 2)
        return (y * dy).sum() + (e * ds).sum()

    got = R.short_conv_adjoint(x, w, b, s, dy, ds, lengths, silu)
    _close(got["dx"], _differences(lambda v: loss(x=v), x))
    _close(got["dweight"], _differences(lambda v: loss(w=v), w))
    _close(got["dbias"], _differences(lambda v: loss(b=v), b))
    _close(got["dstate_in"], _differences(lambda v: loss(s=v), s))


# ------------------------------------------------------------------ norm and rotation
def test_rotation_keeps_products_of_equal_distances():
    rng = np.random.default_rng(3)
    x, y = rng.standard_normal((1, 1, 1, 16)), rng.standard_normal((1, 1, 1, 16))
    f, _ = R.rope_frequencies(16)
    for inter in (False, True):
        at = lambda v, p: R.qk_norm_rope(v, None, f, np.array([[p]]), None, interleaved=inter)[0, 0, 0]
        want = at(x, 5) @ at(y, 2)
        for p in (0, 1000, -77, 2 ** 20):
            assert abs(at(x, p + 3) @ at(y, p) - want) < 1e-9
        assert np.allclose(np.linalg.norm(at(x, 123456)), np.linalg.norm(x))
    # a quarter turn of the first pair
    q = R.qk_norm_rope(np.arange(8.0).reshape(1, 1, 1, 8), None, np.array([np.pi / 2, 0.0]), np.array([[1]]), None)[0, 0, 0]
    assert np.allclose(q, [-2, 1, 0, 3, 4, 5, 6, 7])
    q = R.qk_norm_rope(np.arange(8.0).reshape(1, 1, 1, 8), None, np.array([np.pi / 2, 0.0]), np.array([[1]]), None, interleaved=True)
    assert np.allclose(q[0, 0, 0], [-1, 0, 2, 3, 4, 5, 6, 7])


def test_norms():
    x = np.random.default_rng(4).standard_normal((1, 2, 3, 8)) * 7
    y = R.qk_norm_rope(x, None, None, None, "rms", 0.0)
    assert np.allclose((y ** 2).mean(-1), 1)
    y = R.qk_norm_rope(x, None, None, None, "l2", 0.0)
    assert np.allclose((y ** 2).sum(-1), 1)
    w = np.arange(24.0).reshape(3, 8)
    assert np.allclose(R.qk_norm_rope(x, w, None, None, "l2", 0.0), y * w[None, :, None])


@pytest.mark.parametrize("norm", ["rms", "l2", None])
@pytest.mark.parametrize("rows", [1, 2])
@pytest.mark.parametrize("inter", [False, True])
def test_qk_adjoint_against_differences(norm, rows, inter):
    rng = np.random.default_rng(5)
    x, dy = rng.standard_normal((2, 2, 2, 8)), rng.standard_normal((2, 2, 2, 8))
    w = None if norm is None else 1 + 0.3 * rng.standard_normal((rows, 8))
    f, _ = R.rope_frequencies(4)
    pos = np.array([[3, 900], [0, -5]])

    def loss(x=x, w=w):
        return (R.qk_norm_rope(x, w, f, pos, norm, 1e-3, inter, 1.3) * dy).sum()

    dx, dw = R.qk_norm_rope_adjoint(x, w, f, dy, pos, norm, 1e-3, inter, 1.3)
    _close(dx, _differences(lambda v: loss(x=v), x))
    if w is not None:
        _close(dw, _differences(lambda v: loss(w=v), w))


# ------------------------------------------------------------------ gated recurrence
def _scan(rng, B, H, T, D):
    n = rng.standard_normal
    return n((B, H, T, D)), n((B, H, T, D)), n((B, H, T, D)), rng.uniform(-1, 1, H), n((H, D)), n((B, H, D))


def test_scan_is_the_sum_over_the_past():
    rng = np.random.default_rng(6)
    x, z, i, A, b, s = _scan(rng, 2, 2, 6, 3)
    y, end, before = R.gated_scan(x, z, A, b, s, i, [6, 4])
    g, a, n, _ = R.scan_gates(z, A, b, True)
    assert np.allclose(a, np.exp(-np.exp(A)[None, :, None, None] * np.log1p(np.exp(z + b[None, :, None]))))
    assert np.allclose(a ** 2 + n ** 2, 1)
    G = np.cumsum(g, 2)
    u = n * x / (1 + np.exp(-i))
    for bb, t in ((0, 5), (1, 3)):
        want = np.exp(G[bb, :, t]) * s[bb] + sum(np.exp(G[bb, :, t] - G[bb, :, k]) * u[bb, :, k] for k in range(t + 1))
        assert np.allclose(y[bb, :, t], want) and np.allclose(end[bb], want)
    assert np.all(y[1, :, 4:] == 0) and np.allclose(before[:, :, 1], y[:, :, 0])
    y1, mid, _ = R.gated_scan(x[:, :, :2], z[:, :, :2], A, b, s, i[:, :, :2])
    y2, end2, _ = R.gated_scan(x[:, :, 2:], z[:, :, 2:], A, b, mid, i[:, :, 2:])
    assert np.allclose(np.concatenate((y1, y2), 2)[0], y[0]) and np.allclose(end2[0], end[0])


@pytest.mark.parametrize("gated", [True, False])
@pytest.mark.parametrize("normalize", [True, False])
@pytest.mark.parametrize("lengths", [None, [3, 0]])
def test_scan_adjoint_against_differences(gated, normalize, lengths):
    rng = np.random.default_rng(7)
    x, z, i, A, b, s = _scan(rng, 2, 2, 4, 2)
    i = i if gated else None
    dy, ds = rng.standard_normal(x.shape), rng.standard_normal(s.shape)

    def loss(x=x, z=z, i=i, A=A, b=b, s=s):
        y, e, _ = R.gated_scan(x, z, A, b, s, i, lengths, normalize)
        return (y * dy).sum() + (e * ds).sum()

    got = R.gated_scan_adjoint(x, z, A, b, s, dy, ds, i, lengths, normalize)
    for name, v, arg in (("dx", x, "x"), ("dz", z, "z"), ("dinput_gate", i, "i"), ("dA_log", A, "A"), ("ddt_bias", b, "b"),
                         ("dstate_in", s, "s")):
        if v is not None:
            _close(got[name], _differences(lambda q: loss(**{arg: q}), v), 1e-7)


def test_scan_adjoint_holds_the_clamp():
    rng = np.random.default_rng(8)
    x, z, i, _, b, s = _scan(rng, 1, 3, 3, 2)
    A = np.array([-11.0, 0.0, 21.0])
    got = R.gated_scan_adjoint(x, z, A, b, s, x, None, i)
    assert got["dA_log"][0] == 0 and got["dA_log"][2] == 0 and got["dA_log"][1] != 0
