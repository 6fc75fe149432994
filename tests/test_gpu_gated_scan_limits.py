"""Gated linear recurrence on the GPU at the ends of its gates, element by element against float64 (the limits are those of
test_gpu_gated_scan)."""
import pytest
import torch

import gated_delta_rule_47_amd as kda

from gpu_helpers import DEV
from test_gpu_gated_scan import BF, FP, check, inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("normalize", [True, False])
def test_a_state_dropped_whole_leaves_the_multiplier_s_gradient(normalize, dtype):
    """A gate so open that its g passes fp32 (z of infinity or the type's largest value: drop the state here): dg g has the
    limit 0 there, whatever else the head holds, and every gradient is what a gate of 1e4 gives, bit by bit."""
    B, H, T, D = 2, 2, 150, 10
    most = torch.finfo(dtype).max
    d = inputs(B, H, T, D, dtype, 21)
    # 1e4: a = 0 in float64 too, and nothing overflows anywhere: the definition in float64 has a number there
    near = {**d, "z": d["z"].clone()}
    places = ((0, 0, 17, 3), (0, 1, 0, 0), (1, 0, 149, 9), (1, 1, 64, 4), (0, 0, 63, 5))
    for p in places:
        near["z"][p] = 1e4
    check(B, H, T, D, dtype, d=near, normalize=normalize)
    call = lambda d: kda.gated_scan_fwd(d["x"], d["z"], d["A"], d["b"], d["s"], d["i"], normalize=normalize, want_ckpt=True)
    back = lambda d, c: kda.gated_scan_bwd(d["x"], d["z"], d["A"], d["b"], c, d["dy"], d["ds"], d["i"], normalize=normalize)
    y0, e0, c0 = call(near)
    g0 = back(near, c0)
    for value in (most, float("inf")):
        far = {**near, "z": near["z"].clone()}
        for p in places:
            far["z"][p] = value
        y, e, c = call(far)
        assert torch.equal(y, y0) and torch.equal(e, e0), value
        g = back(far, c)
        for name in g0:
            assert torch.isfinite(g[name]).all(), (name, value)
            assert torch.equal(g[name], g0[name]), (name, value)
    # A multiplier at its clamp's end takes a finite z past fp32 as well
    d["A"] = torch.tensor([19.9, 0.0], device=DEV)
    d["z"][0, 0, 20, 1] = 1e30
    y, e, c = call(d)
    g = back(d, c)
    assert all(torch.isfinite(t).all() for t in (y, e, *g.values()))
    # a NaN among the gates still reaches its channel's parameters
    d["z"][1, 1, 3, 2] = float("nan")
    g = back(d, call(d)[2])
    assert torch.isnan(g["dA_log"][1]) and torch.isfinite(g["dA_log"][0])
    assert torch.isnan(g["ddt_bias"][1, 2]) and torch.isnan(g["ddt_bias"]).sum() == 1


def test_input_scales_next_to_nothing():
    """Decays so close to 1 that 1 - a^2 is 1e-36 and less: n is its root in the adjoint as it is in the forward pass (from
    z' = -87.3 on, e^z' is below fp32's normal numbers and counts as 0)."""
    T, D = 40, 16
    d = inputs(1, 1, T, D, FP, 22, bias=False)
    d["z"] = torch.linspace(-87.0, -81.0, D, device=DEV).expand(1, 1, T, D).contiguous()
    d["A"] = torch.zeros(1, device=DEV)
    check(1, 1, T, D, FP, d=d)
    # the least multiplier: 1 - a^2 below fp32's normal numbers, where n and all that it scales is at most 2^-63 and may be 0
    d["A"] = torch.full((1,), -10.0, device=DEV)
    call = kda.gated_scan_fwd(d["x"], d["z"], d["A"], None, d["s"], d["i"], want_ckpt=True)
    g = kda.gated_scan_bwd(d["x"], d["z"], d["A"], None, call[2], d["dy"], d["ds"], d["i"])
    r = float((d["dy"].abs().sum(2) + d["ds"].abs()).max()) * float(d["x"].abs().max() + 1)
    assert torch.equal(call[0], d["s"].unsqueeze(2).expand_as(call[0]))
    assert all(torch.isfinite(g[n]).all() for n in g)
    n = 2.0 ** -63                                                 # (sqrt(2 e^-91) = 2^-65 is the largest)
    assert g["dx"].abs().max() <= n * r and g["dinput_gate"].abs().max() <= n * r
    # a decay of exactly 1: the term with 1 / n counts as its limit, 0, for inputs of any size
    d["z"] = torch.full_like(d["z"], -200.0)
    d["x"][0, 0, :, 0] = 1e30
    call = kda.gated_scan_fwd(d["x"], d["z"], d["A"], None, d["s"], d["i"], want_ckpt=True)
    g = kda.gated_scan_bwd(d["x"], d["z"], d["A"], None, call[2], d["dy"], d["ds"], d["i"])
    assert all(torch.isfinite(g[n]).all() for n in g)
    assert not (g["dx"].any() or g["dz"].any() or g["dA_log"].any() or g["dinput_gate"].any())


@pytest.mark.parametrize("B,H,T,D,dtype,lengths,backward", [
    # 10 channel tiles: 71 tiles forward and 141 in the adjoint, one line
    (1, 1, 9000, 1200, BF, None, True), (2, 1, 9000, 640, BF, [9000, 4321], True),
    # 66 channel tiles, the adjoint's tiles of four waves: 75
    (1, 6, 2400, 700, FP, None, True),
    # 130 channel tiles, the forward pass's too: 66
    (1, 1, 4200, 8300, FP, None, False),
    # by groups: 547 tiles in 69 of them forward, 1094 in 137 in the adjoint
    (1, 1, 70000, 4, FP, None, True), (2, 1, 70000, 3, BF, [70000, 69000], True)])
def test_lines_of_more_than_64_tiles(B, H, T, D, dtype, lengths, backward):
    """Every token with its inputs and decays that remember tens of tiles, so that a pair left out or taken twice anywhere in a
    line shows; bit by bit the same when it runs again, where other tiles have finished."""
    d, y, end, ckpt = check(B, H, T, D, dtype, lengths, seed=T + D, slow=True, backward=backward)
    lt = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device=DEV)
    args = (d["x"], d["z"], d["A"], d["b"])
    first = None
    for _ in range(3):
        got = kda.gated_scan_fwd(*args, d["s"], d["i"], lt, out=torch.full_like(y, 7.0))
        assert torch.equal(got[0], y) and torch.equal(got[1], end)
        if backward:
            r = kda.gated_scan_bwd(*args, ckpt, d["dy"], d["ds"], d["i"], lt)
            first = first or r
            assert all(torch.equal(r[k], first[k]) for k in r)
