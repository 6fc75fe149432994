"""The layer operators at the ends of their documented ranges: the longest tensors, the slowest decays, the
smallest numbers, gradients in place at every width."""
import pytest
import torch

import gated_delta_rule_47_amd as kda

from gpu_helpers import DEV, say

pytestmark = pytest.mark.gpu

BF, FP = torch.bfloat16, torch.float32


def test_norm_of_as_many_rows_as_an_int_counts():
    """B H T = 2^31 - 2 rows, of which the run that a workgroup takes last ends next to 2^31: every row is written
    and counts in the sums.  The rows are zeros (y = bias there) but for some of the last run, which give what they
    give alone, and whose terms in the sums over rows do not cancel.  Those terms are ones for the bias (whole
    numbers below 2^24: exact); the weight's go through at most 8192 additions in a thread, 256 in its workgroup and
    64 in the parts' sums, each off by 2^-24 at most."""
    T, D, n = 2 ** 31 - 2, 2, 3 * 10 ** 6
    w = torch.tensor([[1.5, -0.5]], device=DEV)
    b = torch.tensor([[2.0, -3.0]], device=DEV)
    x = torch.zeros((1, 1, T, D), dtype=BF, device=DEV)
    x[..., -n:, :].uniform_(0.5, 2.0)
    x[..., -n:, 1].neg_()
    y = torch.full_like(x, 7.0)
    say("norm", tuple(x.shape))
    _, mean, rstd = kda.layer_norm_fwd(x, w, b, out=y)
    last = lambda t: t[:, :, T - n:].contiguous()
    y1, m1, r1 = kda.layer_norm_fwd(last(x), w, b)
    assert torch.equal(last(y), y1) and torch.equal(last(mean), m1) and torch.equal(last(rstd), r1)
    assert torch.all(y[0, 0, :T - n, 0] == 2.0) and torch.all(y[0, 0, :T - n, 1] == -3.0)
    dy = torch.zeros_like(x)
    dy[..., -n:, :] = 1.0
    dx = y.fill_(7.0)
    say("norm bwd", tuple(x.shape))
    _, dw, db = kda.layer_norm_bwd(x, w, mean, rstd, dy, dx_out=dx)
    dx1, _, _ = kda.layer_norm_bwd(last(x), w, m1, r1, last(dy))
    assert torch.equal(last(dx), dx1)
    assert not dx[0, 0, :T - n].any()
    assert torch.all(db == n)
    xh = (last(x).double() - m1.double().unsqueeze(-1)) * r1.double().unsqueeze(-1)
    assert torch.all((dw.double() - xh.sum((0, 2))).abs() <= 8600 * 2.0 ** -24 * xh.abs().sum((0, 2)))
