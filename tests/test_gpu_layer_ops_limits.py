"""The layer operators at the ends of their documented ranges: the longest tensors, the slowest decays, the
smallest numbers, gradients in place at every width."""
import numpy as np
import pytest
import torch

import gated_delta_rule_47_amd as kda
from oracle import layer_ref as R

from gpu_helpers import DEV, host, say, to_dev

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


@pytest.mark.parametrize("H", [256, 2])
@pytest.mark.parametrize("dtype,C", [(FP, 32), (BF, 64)])
def test_slow_decay_over_thousands_of_chunks(dtype, C, H):
    """65536 tokens, whole (256 heads) or in segments (2 heads), in chunks of C, a decay whose power over a chunk
    lies in the middle between two floats: taken as one float it would be off by 2^-25, always to the same side, and
    what the walks carry by 2048 times that, 6e-5 (bf16: 1024 times, 3e-5); o, dq, dk, dv and the states are right
    whether the end state is asked for or not.  Bar of fp32 results: per chunk a carried value takes at most 10
    roundings (the decay and the products, 8 of 4 tokens each or 6 of bf16 parts), each 2^-24 / sqrt(3) RMS and of
    any sign: sqrt(10 * 2048 / 3) 2^-24 = 4.9e-6 of the 2-norm; twice that is allowed.  bf16 results: u = 2^-8."""
    B, T, D = 1, 65536, 8
    heads = [0, H - 1]
    g = np.float32(np.log1p(-(536.5) * 2.0 ** -24) / C)
    power = np.exp(float(C) * float(g))
    assert abs(np.float32(power) - power) > 0.45 * 2.0 ** -24
    for need in (kda.decay_attn_workspace_bytes, kda.decay_attn_bwd_workspace_bytes):
        assert (need(B, H, T, D, D, dtype) == 0) == (H == 256)
    rng = np.random.default_rng(11)
    x = {n: rng.standard_normal((B, 2, T, D)).astype(np.float32) for n in ("q", "k", "v", "d_o")}
    for n in ("k", "d_o"):
        x[n] *= np.float32(T ** -0.5)                             # the state stays of the size of its start
    for n in ("S0", "dS"):
        x[n] = rng.standard_normal((B, 2, D, D)).astype(np.float32)
    d = {}
    for n, a in x.items():
        part = to_dev(a, FP if n in ("S0", "dS") else dtype)
        d[n] = torch.zeros((B, H, *a.shape[2:]), dtype=part.dtype, device=DEV)
        d[n][:, heads] = part
        x[n] = host(part)
    gd = torch.full((H,), float(g), device=DEV)
    say("slow decay", B, H, T, D, dtype)
    o, _ = kda.decay_attn_fwd(d["q"], d["k"], d["v"], gd, d["S0"], output_state=False)
    o2, S = kda.decay_attn_fwd(d["q"], d["k"], d["v"], gd, d["S0"])
    if dtype == FP:                                               # (bf16: the last bits of a product may differ)
        assert torch.equal(o, o2)
    got = kda.decay_attn_bwd(d["q"], d["k"], d["v"], gd, d["S0"], d["d_o"], d["dS"])
    got.update(o=o, o2=o2, state=S)
    ref = R.decay_attn_adjoint(x["q"], x["k"], x["v"], [g, g], x["S0"], x["d_o"], x["dS"])
    ref["o"], ref["state"] = R.decay_attn(x["q"], x["k"], x["v"], [g, g], x["S0"])
    ref["o2"] = ref["o"]
    err = {n: np.linalg.norm(host(got[n][:, heads]) - ref[n]) / np.linalg.norm(ref[n]) for n in ref}
    say("  ", {n: "%.2e" % e for n, e in err.items()})
    for n, e in err.items():
        assert e <= (1e-5 if got[n].dtype == FP else 2.0 ** -8), err


@pytest.mark.parametrize("dtype", [BF, FP])
def test_thousands_of_tokens_with_a_slow_decay(dtype):
    """4096 single tokens with a decay that lies in the middle between two floats: taken as one it would be off by
    2^-25, and the state by 4096 times that, 1.2e-4.  Bar: three roundings a token (the product k v, the sum with
    the decay's low part, the new state), each 2^-24 / sqrt(3) RMS and of any sign: sqrt(4096) 2^-24 = 3.8e-6 of the
    2-norm; twice that is allowed.  Infinities in the state stay where they are."""
    B, H, T, K, V = 1, 2, 4096, 16, 8
    g = np.float32(np.log1p(-(536.5) * 2.0 ** -24))
    assert abs(np.float32(np.exp(float(g))) - np.exp(float(g))) > 0.45 * 2.0 ** -24
    rng = np.random.default_rng(12)
    x = {n: rng.standard_normal((B, H, T, D)) * T ** -0.25 for n, D in (("q", K), ("k", K), ("v", V))}
    d = {n: to_dev(a.astype(np.float32), dtype) for n, a in x.items()}
    S0 = rng.standard_normal((B, H, K, V)).astype(np.float32)
    S, gd = to_dev(S0, FP), torch.full((H,), float(g), device=DEV)
    tok = [[d[n][:, :, t].contiguous() for n in ("q", "k", "v")] for t in range(T)]
    out = [kda.decay_attn_step(*a, gd, S) for a in tok]
    ro, rS = R.decay_attn(host(d["q"]), host(d["k"]), host(d["v"]), [g, g], S0)
    norm2 = lambda a, b: np.linalg.norm(a - b) / np.linalg.norm(b)
    e, eo = norm2(host(S), rS), norm2(host(torch.stack(out, 2)), ro)
    say("  state %.2e, o %.2e" % (e, eo))
    assert e <= 7.6e-6 and eo <= (2.0 ** -8 if dtype == BF else 7.6e-6 + 2e-6)      # o: and a sum of 16 products
    S[0, 0, 3, 2], S[0, 1, 5, 1] = float("inf"), -float("inf")
    for gg in (0.0, float(g), -3.0):
        kda.decay_attn_step(*tok[0], torch.full((H,), gg, device=DEV), S)
        assert S[0, 0, 3, 2] == float("inf") and S[0, 1, 5, 1] == -float("inf")
        assert int(torch.isfinite(S).sum()) == S.numel() - 2


@pytest.mark.parametrize("dtype,D", [(BF, 40), (BF, 4100), (BF, 16384), (BF, 16392), (FP, 8192), (FP, 8200), (FP, 20001)])
def test_norm_gradient_in_place_of_its_cotangent(dtype, D):
    """dx written over dy, with the sums, in rows of a wave, of a workgroup, and wider: the same as apart."""
    x, dy = (torch.randn(2, 2, 9, D, device=DEV).to(dtype) for _ in range(2))
    w = torch.randn(2, D, device=DEV)
    _, mean, rstd = kda.layer_norm_fwd(x, w)
    want = kda.layer_norm_bwd(x, w, mean, rstd, dy)
    got = kda.layer_norm_bwd(x, w, mean, rstd, dy, dx_out=dy)
    assert got[0] is dy
    for a, b in zip(got, want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("D", [32, 31])
def test_every_code_under_every_scale(D):
    """Each of the 256 codes under each of the 256 scale bytes, in groups read eight at a time and one by one.  fp32
    holds every value (the smallest is 2^-136, the largest 448 2^128 is infinite); bf16 rounds those below 2^-130
    that are no multiple of 2^-133 to the nearest, ties to even."""
    codes = np.tile(np.arange(256, dtype=np.uint8), (256, 1))
    codes = np.concatenate([codes, np.zeros((256, -256 % D), np.uint8)], 1).reshape(-1, D)
    scales = np.repeat(np.arange(256, dtype=np.uint8), len(codes) // 256)[:, None]
    with np.errstate(over="ignore"):
        want = torch.from_numpy(R.ckpt_unpack(codes, scales).astype(np.float32))
    c, s = torch.from_numpy(codes).to(DEV), torch.from_numpy(scales).to(DEV)
    ok = scales[:, 0] < 255                                       # (255 is no scale that a packed group has)
    for dtype in (FP, BF):
        got = kda.ckpt_unpack(c, s, dtype).cpu()[ok]
        ref = want.to(dtype)[ok]
        nan = torch.isnan(ref)
        assert torch.equal(torch.isnan(got), nan)
        assert torch.equal(got[~nan], ref[~nan]), dtype
    big = np.abs(want.numpy())[ok]
    exact = (want.to(BF).float() == want).numpy()[ok]
    fin = np.isfinite(big) & (big > 0)
    assert exact[fin & (big >= 2.0 ** -130)].all() and not exact[fin & (big < 2.0 ** -130) & (big > 2.0 ** -131)].all()


@pytest.mark.parametrize("dtype", [BF, FP])
def test_smallest_activations_in_8_bits(dtype):
    """Subnormal and smallest normal values through pack and unpack: codes as defined, fp32 restored to the value of
    its code, bf16 to that value rounded to nearest even."""
    rng = np.random.default_rng(5)
    x = (rng.standard_normal((64, 64)) * 2.0 ** rng.integers(-140, -115, (64, 1))).astype(np.float32)
    d = torch.from_numpy(x).to(dtype).to(DEV)
    codes, scales = kda.ckpt_pack(d)
    rc, rs = R.ckpt_pack(d.float().cpu().numpy())
    assert np.array_equal(codes.cpu().numpy(), rc) and np.array_equal(scales.cpu().numpy(), rs)
    val = torch.from_numpy(R.ckpt_unpack(rc, rs).astype(np.float32)).to(dtype)
    assert torch.equal(kda.ckpt_unpack(codes, scales, dtype).cpu(), val)


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("T", [1, 90, 1100])
def test_gradients_along_themselves_against_differences(T, dtype):
    """The float64 definition's loss along the direction of each computed gradient g: where t is the true one its
    slope there is <t, g> / |g|, which differs from |g| by at most |g - t|.  That is u = 2^-8 of |g| in bf16 (scores,
    state and the output, each rounded once, see test_gpu_decay_attn.py) and 2e-5 in fp32.  The loss is linear in q,
    k, v and the start state each, so central differences are exact but for the rounding of two sums."""
    B, H, K, V = 1, 2, 16, 32
    rng = np.random.default_rng(T)
    x = {n: rng.standard_normal((B, H, T, D)) for n, D in (("q", K), ("k", K), ("v", V), ("d_o", V))}
    x["q"] /= K ** 0.5
    d = {n: to_dev(a.astype(np.float32), dtype) for n, a in x.items()}
    x = {n: host(t) for n, t in d.items()}
    g = np.float32([-0.3, -0.01])
    S0, dS = (rng.standard_normal((B, H, K, V)).astype(np.float32) for _ in range(2))
    got = kda.decay_attn_bwd(d["q"], d["k"], d["v"], to_dev(g, FP), to_dev(S0, FP), d["d_o"], to_dev(dS, FP))
    base = {"dq": x["q"], "dk": x["k"], "dv": x["v"], "dstate_in": S0.astype(np.float64)}

    def loss(at):
        o, S = R.decay_attn(at["dq"], at["dk"], at["dv"], g, at["dstate_in"])
        return (o * x["d_o"]).sum() + (S * dS).sum()

    for n in base:
        a = host(got[n])
        norm = np.linalg.norm(a)
        up, dn = (loss({**base, n: base[n] + h * a / norm}) for h in (0.5, -0.5))
        bar = 2.0 ** -8 if dtype == BF and n != "dstate_in" else 2e-5
        say("  %-9s |g| %.6e, slope %.6e, off by %.1e (bar %.1e)" % (n, norm, up - dn, abs(up - dn - norm) / norm, bar))
        assert abs(up - dn - norm) <= bar * norm + 1e-13 * (abs(up) + abs(dn)), n


@pytest.mark.parametrize("K,V", [(8, 8), (128, 128)])
def test_as_many_heads_as_a_call_takes(K, V):
    """2^20 heads of one and of two tokens, forward, single token and backward: the last head, one in the middle and
    the first are what they are alone (the plans differ by the number of heads, but not for so few tokens: bit for
    bit but for the value tiles' width, which changes no sum)."""
    B, H = 1024, 1024
    pick = lambda t: torch.stack([t[0, 0], t[511, 700], t[-1, -1]]).unsqueeze(0).contiguous()
    for T in (1, 2):
        q, k, v, d_o = (torch.randn(B, H, T, D, device=DEV, dtype=BF) for D in (K, K, V, V))
        g = torch.full((H,), -0.25, device=DEV)
        say("heads", B * H, K, V, T)
        o, S = kda.decay_attn_fwd(q, k, v, g)
        o1, S1 = kda.decay_attn_fwd(pick(q), pick(k), pick(v), g[:3])
        assert torch.equal(pick(o), o1) and torch.equal(pick(S), S1)
        if T == 1:
            one = [t[:, :, 0].contiguous() for t in (q, k, v)]
            o = kda.decay_attn_step(*one, g, S)
            o1 = kda.decay_attn_step(*(pick(t) for t in one), g[:3], S1)
            assert torch.equal(pick(o), o1) and torch.equal(pick(S), S1)
        del o, S
        got = kda.decay_attn_bwd(q, k, v, g, None, d_o)
        one = kda.decay_attn_bwd(pick(q), pick(k), pick(v), g[:3], None, pick(d_o))
        for n in got:
            assert torch.equal(pick(got[n]), one[n]), n
        del got


def test_norm_of_as_many_heads_as_a_call_takes():
    """2^20 heads, 2^28 weights: dw and db of a head with one row are its terms themselves."""
    B, H, T, D = 1, 2 ** 20, 1, 256
    x, dy = (torch.randn(B, H, T, D, device=DEV, dtype=BF) for _ in range(2))
    w = torch.randn(H, D, device=DEV)
    y, mean, rstd = kda.layer_norm_fwd(x, w)
    dx, dw, db = kda.layer_norm_bwd(x, w, mean, rstd, dy)
    xh = (x.float() - mean.unsqueeze(-1)) * rstd.unsqueeze(-1)
    assert torch.equal(db, dy[0, :, 0].float())
    assert torch.allclose(dw, (dy.float() * xh)[0, :, 0], rtol=2.0 ** -22, atol=0)       # three roundings
    last = lambda t: t[:, -1:].contiguous()
    y1, m1, r1 = kda.layer_norm_fwd(last(x), w[-1:])
    assert torch.equal(last(y), y1) and torch.equal(last(mean), m1) and torch.equal(last(rstd), r1)
    dx1, dw1, db1 = kda.layer_norm_bwd(last(x), w[-1:], m1, r1, last(dy))
    assert torch.equal(last(dx), dx1) and torch.equal(dw[-1:], dw1) and torch.equal(db[-1:], db1)


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("T", [70, 2100])
def test_one_tensor_for_several_inputs(T, dtype):
    """The same tensor as q, k, v and d_o, the same state as start and as cotangent: what copies of it give."""
    x = torch.randn(1, 2, T, 64, device=DEV).to(dtype)
    S = torch.randn(1, 2, 64, 64, device=DEV)
    g = torch.tensor([-0.2, -0.01], device=DEV)
    c = [x.clone() for _ in range(4)]
    for a, b in zip(kda.decay_attn_fwd(x, x, x, g, S), kda.decay_attn_fwd(*c[:3], g, S.clone())):
        assert torch.equal(a, b)
    a = kda.decay_attn_bwd(x, x, x, g, S, x, S)
    b = kda.decay_attn_bwd(*c[:3], g, S.clone(), c[3], S.clone())
    for n in a:
        assert torch.equal(a[n], b[n]), n
    p = kda.ckpt_pack(x)
    a, b = kda.decay_attn_bwd(p, p, p, g, S, x, S), kda.decay_attn_bwd(*(kda.ckpt_pack(t) for t in c[:3]), g, S, x, S)
    for n in a:
        assert torch.equal(a[n], b[n]), n
    y, mean, rstd = kda.layer_norm_fwd(x)
    for a, b in zip(kda.layer_norm_bwd(x, None, mean, rstd, x), kda.layer_norm_bwd(x, None, mean, rstd, c[0])):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("T", [200, 2200])
def test_non_finite_tokens_reach_their_block_and_what_depends_on_them(T, dtype):
    """A non-finite token in one head: outputs of earlier blocks of 64 tokens (in a backward pass the gradients that
    flow the other way: later ones) and the other head are those of the clean call, bit for bit."""
    B, H, D, t = 1, 2, 64, 130
    d = {n: torch.randn(B, H, T, D, device=DEV).to(dtype) for n in ("q", "k", "v", "d_o")}
    S, dS = (torch.randn(B, H, D, D, device=DEV) for _ in range(2))
    g = torch.tensor([-0.05, -0.2], device=DEV)
    fwd = lambda a: kda.decay_attn_fwd(a["q"], a["k"], a["v"], g, S)
    bwd = lambda a: kda.decay_attn_bwd(a["q"], a["k"], a["v"], g, S, a["d_o"], dS)
    o, E = fwd(d)
    r = bwd(d)
    for name, bad in (("q", float("nan")), ("k", float("inf")), ("v", float("nan")), ("d_o", -float("inf"))):
        a = dict(d, **{name: d[name].clone()})
        a[name][0, 0, t] = bad
        o2, E2 = fwd(a)
        assert torch.equal(o2[0, 1], o[0, 1]) and torch.equal(E2[0, 1], E[0, 1])
        assert torch.equal(o2[0, 0, :128], o[0, 0, :128])
        if name == "q":                                           # read by its own token only
            assert torch.equal(o2[0, 0, 192:], o[0, 0, 192:]) and torch.equal(E2, E)
            assert torch.isnan(o2[0, 0, t]).all()
        r2 = bwd(a)
        for n in r:
            assert torch.equal(r2[n][0, 1], r[n][0, 1]), (name, n)
        if name in ("k", "v"):                                    # dq of its block and later ones, its own dk or dv
            assert torch.equal(r2["dq"][0, 0, :128], r["dq"][0, 0, :128])
            for n in ("dk", "dv"):
                assert torch.equal(r2[n][0, 0, :128], r[n][0, 0, :128]) and torch.equal(r2[n][0, 0, 192:], r[n][0, 0, 192:])
            assert torch.equal(r2["dstate_in"], r["dstate_in"])
        else:                                                     # dk and dv of its block and earlier ones
            for n in ("dk", "dv"):
                assert torch.equal(r2[n][0, 0, 192:], r[n][0, 0, 192:])
            if name == "d_o":
                assert torch.equal(r2["dq"][0, 0, :128], r["dq"][0, 0, :128])
                assert torch.equal(r2["dq"][0, 0, 192:], r["dq"][0, 0, 192:])
            else:
                assert torch.equal(r2["dq"], r["dq"])
