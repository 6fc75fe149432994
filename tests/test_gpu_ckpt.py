"""8-bit activations on the GPU: codes, scales and restored values equal those of the definition."""
import numpy as np
import pytest
import torch

import gated_delta_rule_47_amd as kda
from oracle import layer_ref as R

from gpu_helpers import DEV, say

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float32


def run(x, shift=0):
    """x: float32 or bf16 tensor on the CPU, (rows, D)."""
    say("ckpt", tuple(x.shape), x.dtype, shift)
    d = torch.empty(x.numel() + shift, dtype=x.dtype, device=DEV)[shift:].view(x.shape).copy_(x)
    codes, scales = kda.ckpt_pack(d)
    rc, rs = R.ckpt_pack(x.float().numpy())
    nan = (rc & 127) == 127
    got = codes.cpu().numpy()
    assert np.array_equal(scales.cpu().numpy(), rs)
    assert np.array_equal(got[~nan], rc[~nan]) and np.all((got[nan] & 127) == 127)
    val = R.ckpt_unpack(rc, rs)
    y = torch.empty(x.numel() + shift, dtype=x.dtype, device=DEV)[shift:].view(x.shape)
    kda.ckpt_unpack(codes, scales, x.dtype, out=y)
    y = y.float().cpu().double().numpy()
    big = np.abs(val) >= (2.0 ** -126 if x.dtype == BF else 2.0 ** -126)
    assert np.array_equal(y[big & ~nan], val[big & ~nan]) and np.all(np.isnan(y[nan]))
    assert np.all(np.abs(y - val)[~big & ~nan] <= 2.0 ** -133)     # half a step of bf16's subnormals, and below


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("D", [1, 3, 7, 8, 9, 15, 16, 24, 31, 32, 64, 96, 128, 512, 1024])
@pytest.mark.parametrize("rows", [1, 37])
def test_widths(rows, D, dtype):
    rng = np.random.default_rng(D)
    x = (rng.standard_normal((rows, D)) * 2.0 ** rng.integers(-40, 40, (rows, 1))).astype(np.float32)
    run(torch.from_numpy(x).to(dtype))
    run(torch.from_numpy(x).to(dtype), shift=1)


@pytest.mark.parametrize("dtype", [BF, FP])
def test_ties_and_borders(dtype):
    """Every code's value, the middles between neighbours, and amax at and next to 448 2^e."""
    v = R.e4m3_values()[:127]
    mids = (v[1:] + v[:-1]) / 2
    x = np.concatenate([v, mids, -v, -mids])
    x = np.concatenate([x, np.zeros(-len(x) % 31)])
    x = np.concatenate([x.reshape(-1, 31), np.full((len(x) // 31, 1), 448.0)], 1)     # every group's scale is 1
    run(torch.from_numpy(x.astype(np.float32)).to(dtype))
    edge = np.zeros((6, 32), np.float32)
    edge[:, 0] = (448.0, 450.0, 447.0, 1.75, 1.7578125, 1.7421875)
    edge[:, 1] = 0.3
    run(torch.from_numpy(edge).to(dtype))


@pytest.mark.parametrize("dtype", [BF, FP])
def test_extremes(dtype):
    x = np.zeros((8, 64), np.float32)
    x[0, :4] = (np.inf, -np.inf, np.nan, 2.0)
    x[1, 0], x[1, 1] = 3.0e38, -1.0e38
    x[2, 0], x[2, 1] = 2.0 ** -126, -(2.0 ** -127)
    x[3, :] = np.inf
    x[4, 0] = -0.0
    x[5, 0] = 2.0 ** -133
    x[6, :] = np.linspace(-1, 1, 64)
    run(torch.from_numpy(x).to(dtype))


def test_many_rows_and_none():
    rng = np.random.default_rng(3)
    x = torch.from_numpy(rng.standard_normal((70001, 32)).astype(np.float32)).to(BF)
    run(x)
    c, s = kda.ckpt_pack(torch.empty(0, 64, device=DEV))
    assert c.shape == (0, 64) and s.shape == (0, 2) and kda.ckpt_unpack(c, s, FP).shape == (0, 64)


def test_head_major_shape():
    x = torch.randn(2, 3, 5, 64, device=DEV, dtype=BF)
    c, s = kda.ckpt_pack(x)
    assert c.shape == x.shape and s.shape == (2, 3, 5, 2)
    y = kda.ckpt_unpack(c, s)
    assert y.dtype == BF and torch.all((y.float() - x.float()).abs() <= x.float().abs() * 2.0 ** -4 + 2.0 ** -10 * 2.0 ** -5)
