"""The operators between a layer's projections and its mixer run together as a layer runs them, on other streams, in graphs
and at the same time."""
import numpy as np
import pytest
import torch

import gated_delta_rule_47_amd as kda
from oracle import layer_ref as L
from oracle import sequence_ref as R

from gpu_helpers import DEV, host, say, to_dev

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float32


def rel(got, ref):
    return np.linalg.norm(host(got) - ref) / np.linalg.norm(ref)


def attention(dtype, B=2, T=150, H=2, D=32, seed=0):
    """Inputs of one linear-attention layer behind its fused projection: three convolutions side by side, norm and rotation
    of queries and keys, attention with a decay per head."""
    rng = np.random.default_rng(seed)
    C = 3 * H * D
    p = {"x": to_dev(rng.standard_normal((B, T, C)), dtype), "w": to_dev(rng.standard_normal((C, 4)) * 0.5, FP),
         "b": to_dev(0.1 * rng.standard_normal(C), FP), "g": to_dev([-0.05, -0.2], FP),
         "qw": to_dev(1 + 0.1 * rng.standard_normal((1, D)), FP), "kw": to_dev(1 + 0.1 * rng.standard_normal((1, D)), FP),
         "do": to_dev(rng.standard_normal((B, H, T, D)), dtype), "f": kda.rope_frequencies(D, device=DEV)[0]}
    return p


def forward(p, H, D, lengths=None):
    y, conv_state = kda.short_conv_fwd(p["x"], p["w"], p["b"], lengths=lengths, heads=3 * H, out=torch.zeros(
        (p["x"].shape[0], 3 * H, p["x"].shape[1], D), dtype=p["x"].dtype, device=DEV))
    tok = y.transpose(1, 2)                                        # (B, T, 3 H, D) views: the norm takes any strides
    q, k = kda.qk_norm_rope_fwd(tok[:, :, :H], tok[:, :, H:2 * H], p["f"], q_weight=p["qw"], k_weight=p["kw"])
    v = y[:, 2 * H:].contiguous()
    o, state = kda.decay_attn_fwd(q, k, v, p["g"], lengths=lengths, out=torch.zeros_like(v))
    return y, q, k, v, o, state, conv_state


def backward(p, H, D, y, q, k, v):
    a = kda.decay_attn_bwd(q, k, v, p["g"], None, p["do"])
    dy = torch.empty_like(y)
    tok, dtok = y.transpose(1, 2), dy.transpose(1, 2)
    n = kda.qk_norm_rope_bwd(tok[:, :, :H], tok[:, :, H:2 * H], p["f"], a["dq"], a["dk"], q_weight=p["qw"], k_weight=p["kw"],
                             dq_out=dtok[:, :, :H], dk_out=dtok[:, :, H:2 * H])
    dy[:, 2 * H:] = a["dv"]
    c = kda.short_conv_bwd(p["x"], p["w"], p["b"], None, dy)
    return {"dx": c["dx"], "dw": c["dweight"], "db": c["dbias"], "dqw": n["dq_weight"], "dkw": n["dk_weight"]}


@pytest.mark.parametrize("dtype", [BF, FP])
def test_linear_attention_layer_and_its_gradients(dtype):
    """bf16: four operators, each off by a rounding of its inputs and outputs and the attention by three (2^-8 each, not in
    line): sqrt(4 + 3) 2^-8 = 1.1e-2, backward twice as many: 1.5e-2, which a norm's cancellation may double.  fp32: 1e-5 is
    over a hundred roundings of 2^-24 in line."""
    B, T, H, D = 2, 150, 2, 32
    p = attention(dtype)
    y, q, k, v, o, state, _ = forward(p, H, D)
    g = backward(p, H, D, y, q, k, v)
    torch.cuda.synchronize()
    P = {n: host(t) for n, t in p.items() if n != "f"}
    f = p["f"].cpu().numpy()
    yr, _ = R.short_conv(P["x"], P["w"], P["b"], heads=3 * H)
    tok = yr.transpose(0, 2, 1, 3)
    qr, kr = (R.qk_norm_rope(tok[:, :, s], P[w], f) for s, w in ((slice(0, H), "qw"), (slice(H, 2 * H), "kw")))
    ref, sr = L.decay_attn(qr, kr, yr[:, 2 * H:], P["g"])
    bar = 1.1e-2 if dtype == BF else 1e-5
    assert rel(o, ref) <= bar and rel(state, sr) <= bar
    a = L.decay_attn_adjoint(qr, kr, yr[:, 2 * H:], P["g"], None, P["do"])
    dqx, dqw = R.qk_norm_rope_adjoint(tok[:, :, :H], P["qw"], f, a["dq"])
    dkx, dkw = R.qk_norm_rope_adjoint(tok[:, :, H:2 * H], P["kw"], f, a["dk"])
    dyr = np.concatenate((dqx.transpose(0, 2, 1, 3), dkx.transpose(0, 2, 1, 3), a["dv"]), 1)
    c = R.short_conv_adjoint(P["x"], P["w"], P["b"], None, dyr)
    for name, r in (("dx", c["dx"]), ("dw", c["dweight"]), ("db", c["dbias"]), ("dqw", dqw), ("dkw", dkw)):
        assert rel(g[name], r) <= (3e-2 if dtype == BF else 1e-5), (name, rel(g[name], r))


def test_serving_continues_a_padded_batch_of_prompts():
    """Prompts of different lengths, then tokens one by one with the states kept, against the whole sequences: the same
    operators in other pieces, a bf16 rounding apart (the bar of the layer test)."""
    B, T, H, D, more = 3, 60, 2, 32, 5
    p = attention(BF, B, T, H, D, seed=3)
    lens = [40, 0, 55]
    lt = torch.tensor(lens, dtype=torch.int32, device=DEV)
    _, _, _, _, o, state, conv = forward(p, H, D, lt)
    whole = forward(p, H, D)[4]
    for b, n in enumerate(lens):
        assert torch.equal(o[b, :, n:], torch.zeros_like(o[b, :, n:]))
        if n:
            assert rel(o[b, :, :n], host(whole[b, :, :n])) <= 1.1e-2
    pos = lt.clone()
    rows = torch.arange(B, device=DEV)
    for _ in range(more):
        xt = p["x"][rows, pos.long()]
        yt = kda.short_conv_step(xt, p["w"], p["b"], conv).view(B, 1, 3 * H, D)
        q, k = kda.qk_norm_rope_fwd(yt[:, :, :H], yt[:, :, H:2 * H], p["f"], pos.view(B, 1), q_weight=p["qw"], k_weight=p["kw"])
        ot = kda.decay_attn_step(q.view(B, H, D), k.view(B, H, D), yt[:, 0, 2 * H:].contiguous(), p["g"], state)
        want = whole[rows, :, pos.long()]
        assert rel(ot, host(want)) <= 1.5e-2
        pos += 1


@pytest.mark.parametrize("dtype", [BF, FP])
def test_recurrent_block_and_its_gradients(dtype):
    """A convolution in front of the recurrence, the norm of its read behind it; same bars."""
    B, T, D = 2, 300, 64
    rng = np.random.default_rng(4)
    x, z, i, dn = (to_dev(rng.standard_normal((B, T, D)), dtype) for _ in range(4))
    w, cb = to_dev(rng.standard_normal((D, 4)) * 0.5, FP), to_dev(0.1 * rng.standard_normal(D), FP)
    A, b = to_dev([0.3], FP), to_dev(rng.uniform(-5, -1, (1, D)), FP)
    nw = to_dev(1 + 0.1 * rng.standard_normal((1, D)), FP)
    z4, i4, dn4 = z.view(B, 1, T, D), i.view(B, 1, T, D), dn.view(B, 1, T, D)
    u, _ = kda.short_conv_fwd(x, w, cb)
    h, _, ckpt = kda.gated_scan_fwd(u, z4, A, b, input_gate=i4, want_ckpt=True)
    n, mean, rstd = kda.layer_norm_fwd(h, nw)
    dh, dnw, _ = kda.layer_norm_bwd(h, nw, mean, rstd, dn4)
    s = kda.gated_scan_bwd(u, z4, A, b, ckpt, dh, input_gate=i4)
    c = kda.short_conv_bwd(x, w, cb, None, s["dx"])
    torch.cuda.synchronize()
    ur, _ = R.short_conv(host(x), host(w), host(cb))
    hr, _, _ = R.gated_scan(ur, host(z4), host(A), host(b), None, host(i4))
    nr, mr, rr = L.layer_norm(hr, host(nw))
    dhr, dnwr, _ = L.layer_norm_adjoint(hr, host(nw), mr, rr, host(dn4))
    sr = R.gated_scan_adjoint(ur, host(z4), host(A), host(b), None, dhr, None, host(i4))
    cr = R.short_conv_adjoint(host(x), host(w), host(cb), None, sr["dx"])
    for name, got, ref in (("n", n, nr), ("dnw", dnw, dnwr), ("dz", s["dz"], sr["dz"]), ("di", s["dinput_gate"], sr["dinput_gate"]),
                           ("dA", s["dA_log"], sr["dA_log"]), ("db", s["ddt_bias"], sr["ddt_bias"]), ("dx", c["dx"], cr["dx"]),
                           ("dw", c["dweight"], cr["dweight"])):
        assert rel(got, ref) <= (3e-2 if dtype == BF else 2e-5), (name, rel(got, ref))


def _everything(p, H, D, scan, ws):
    """One pass through every entry point, outputs and workspaces given where the captured call needs them."""
    y, q, k, v, o, state, conv = forward(p, H, D)
    out = dict(backward(p, H, D, y, q, k, v), o=o, state=state, conv=conv)
    h, end, ckpt = kda.gated_scan_fwd(*scan[:5], input_gate=scan[5], want_ckpt=True, workspace=ws[0])
    out.update({"scan_" + n: t for n, t in kda.gated_scan_bwd(*scan[:4], ckpt, h, end, scan[5], workspace=ws[1]).items()}, h=h, end=end)
    return out


def _scan_inputs(seed, T=700):
    rng = np.random.default_rng(seed)
    n = lambda *s: to_dev(rng.standard_normal(s), BF)
    return (n(2, 2, T, 32), n(2, 2, T, 32), to_dev([0.2, -0.3], FP), to_dev(rng.uniform(-6, 0, (2, 32)), FP),
            to_dev(rng.standard_normal((2, 2, 32)), FP), n(2, 2, T, 32))


def _scan_ws(T=700):
    return tuple(torch.empty(f(2, 2, T, 32), dtype=torch.uint8, device=DEV)
                 for f in (kda.gated_scan_workspace_bytes, kda.gated_scan_bwd_workspace_bytes))


def test_another_stream_and_graph_replays():
    """Captured once, replayed with eager work and synchronizations between, new inputs among them; two graphs share one
    workspace, replayed one behind the other."""
    H, D = 2, 32
    ws = _scan_ws()
    sets = [(attention(BF, seed=s), _scan_inputs(s)) for s in (5, 6)]
    want = [_everything(p, H, D, sc, ws) for p, sc in sets]
    torch.cuda.synchronize()
    want = [{n: t.clone() for n, t in w.items()} for w in want]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = _everything(*(sets[0][0], H, D, sets[0][1], ws))
    side.synchronize()
    for n in want[0]:
        assert torch.equal(got[n], want[0][n]), n
    graphs = []
    for p, sc in sets:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            r = _everything(p, H, D, sc, ws)
        graphs.append((g, r))
    for rep in range(4):
        for (g, r), w in zip(graphs, want):
            for t in r.values():
                t.fill_(float("nan"))
            torch.cuda.synchronize()
            g.replay()
            torch.cuda.synchronize()
            say("replay", rep)
            for n in w:
                assert torch.equal(r[n], w[n]), (rep, n)
        _ = (sets[0][0]["x"].float() * 2).sum().item()
    for g, _ in graphs:                                            # back to back, one stream
        g.replay()
    torch.cuda.synchronize()
    for (_, r), w in zip(graphs, want):
        assert all(torch.equal(r[n], w[n]) for n in w)
    sets[0][0]["x"].copy_(sets[1][0]["x"])                         # new data at the captured addresses
    for a, b in zip(sets[0][1], sets[1][1]):
        a.copy_(b)
    fresh = _everything(sets[0][0], H, D, sets[0][1], ws)
    graphs[0][0].replay()
    torch.cuda.synchronize()
    assert all(torch.equal(graphs[0][1][n], fresh[n]) for n in fresh)


def test_two_calls_at_once():
    """Two long recurrences on two streams, each with its workspace, whose workgroups share the chip: both end and give what
    they give alone, forward and backward."""
    T = 6000
    calls = []
    for seed in (1, 2):
        sc = _scan_inputs(seed, T)
        ws = _scan_ws(T)
        h, end, ckpt = kda.gated_scan_fwd(*sc[:5], input_gate=sc[5], want_ckpt=True, workspace=ws[0])
        r = kda.gated_scan_bwd(*sc[:4], ckpt, h, end, sc[5], workspace=ws[1])
        calls.append((sc, ws, h, end, r, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for rep in range(5):
        got = []
        for sc, ws, _, _, _, s in calls:
            with torch.cuda.stream(s):
                h, end, ckpt = kda.gated_scan_fwd(*sc[:5], input_gate=sc[5], want_ckpt=True, workspace=ws[0])
                got.append((h, end, kda.gated_scan_bwd(*sc[:4], ckpt, h, end, sc[5], workspace=ws[1])))
        torch.cuda.synchronize()
        say("pair", rep)
        for (_, _, h, end, r, _), (h2, end2, r2) in zip(calls, got):
            assert torch.equal(h, h2) and torch.equal(end, end2) and all(torch.equal(r[n], r2[n]) for n in r)


def test_tensors_off_the_gpu_are_refused():
    x, w = torch.zeros(1, 4, 8, device=DEV), torch.zeros(8, 4)
    with pytest.raises(ValueError):
        kda.short_conv_fwd(x, w)
    with pytest.raises(ValueError):
        kda.qk_norm_rope_fwd(x.view(1, 4, 1, 8), None, kda.rope_frequencies(8)[0])
    with pytest.raises(ValueError):
        kda.gated_scan_fwd(x.view(1, 1, 4, 8), x.view(1, 1, 4, 8), torch.zeros(1))
