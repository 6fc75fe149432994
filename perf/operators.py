"""The workloads the layer operators around the delta rule are measured on.

Three groups, as a linear-attention layer uses them together:

  attn     linear attention with a constant decay per head, S_t = exp(g_h) S_{t-1} + k_t v_t^T,
           o_t = scale S_t^T q_t: prompts ("attn_fwd"), single tokens ("attn_step"), training
           ("attn_bwd")
  norm     layer norm over the last axis with a weight and bias row per head: "norm_fwd", and
           "norm_bwd" with the reduction of the weight's and the bias' gradient
  ckpt     activations kept for the backward pass in 8 bits (e4m3 codes, one power-of-two scale per
           group of at most 32 channels): "ckpt" stores and restores, "attn_bwd" / "norm_bwd" with
           ckpt = True read them as they are kept

With `own` false, run() computes the plain forms in float32; with `own` true it makes the calls a
user makes.  Layouts are head-major and contiguous: (B, H, T, D), states (B, H, K, V) float32.
"""
import math

import torch

own = False

DEV = "cuda:0"
EPS = 1e-5
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _attn(name, op, B, H, T, K, V, dtype, ragged=False, ckpt=False):
    return {"name": name, "op": op, "B": B, "H": H, "T": T, "K": K, "V": V, "dtype": dtype, "ragged": ragged,
            "ckpt": ckpt}


def _norm(name, op, B, H, T, D, dtype, ckpt=False):
    return {"name": name, "op": op, "B": B, "H": H, "T": T, "D": D, "dtype": dtype, "ckpt": ckpt}


def listed():
    return [
        # prefill of four long contexts, every head of a large layer (the long workload's shape)
        _attn("fwd long", "attn_fwd", 4, 32, 16384, 128, 128, "bf16"),
        # one prompt on few heads (a head-parallel shard): the time axis has to give the parallelism
        _attn("fwd one prompt", "attn_fwd", 1, 4, 30011, 128, 128, "bf16"),
        # a padded batch of prompts of different lengths, one of them empty (the nano layer's shape)
        _attn("fwd padded batch", "attn_fwd", 8, 8, 4096, 64, 64, "bf16", ragged=True),
        # a short fp32 sequence of a single layer: latency
        _attn("fwd short f32", "attn_fwd", 1, 8, 257, 64, 64, "f32"),
        # decode of four sequences (latency) and of a full serving batch (state traffic)
        _attn("step few", "attn_step", 4, 32, 1, 128, 128, "bf16"),
        _attn("step many", "attn_step", 192, 32, 1, 128, 128, "bf16"),
        # training step of the nano layer, and of the fp32 adjoint workload's heads at an odd length
        _attn("bwd bf16", "attn_bwd", 8, 8, 4096, 64, 64, "bf16"),
        _attn("bwd f32", "attn_bwd", 1, 16, 8191, 128, 128, "f32"),
        # training on long sequences, where q, k and v are what fills the memory: kept in 8 bits
        _attn("bwd from 8 bits", "attn_bwd", 2, 32, 8192, 128, 128, "bf16", ckpt=True),
        # the same sequences' activations stored in 8 bits and restored
        _norm("store 8 bits", "ckpt", 2, 32, 8192, 128, "bf16"),
        # the nano model's rows of 512 channels before a layer
        _norm("norm rows", "norm_fwd", 1, 1, 32768, 512, "bf16"),
        # the per-head norm of the read of the long-sequence training step, backward
        _norm("norm bwd heads", "norm_bwd", 2, 32, 8192, 128, "bf16"),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["attn_fwd", "attn_fwd", "attn_bwd", "attn_bwd", "attn_step", "norm_fwd", "norm_bwd", "ckpt"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op.startswith("attn"):
        K = rng.choice([8, 16, 32, 64, 64, 128, 128])
        V = rng.choice([8, 16, 32, 64, 64, 128, 128])
        H = _log_int(rng, 1, 40)
        if op == "attn_step":
            B = _log_int(rng, 1, 192)
            return {k: v for k, v in _attn("", op, B, H, 1, K, V, dtype).items() if k != "name"}
        T = _log_int(rng, 1, 32768)
        B = _log_int(rng, 1, 16)
        most = 1 << (28 if op == "attn_fwd" else 26)        # elements of q, k, v and o together
        while B * H * T * 2 * (K + V) > most and B * H > 1:
            B, H = (max(1, B // 2), H) if B >= H else (B, max(1, H // 2))
        ragged = rng.random() < 0.4
        ckpt = op == "attn_bwd" and rng.random() < 0.3
        return {k: v for k, v in _attn("", op, B, H, T, K, V, dtype, ragged, ckpt).items() if k != "name"}
    D = _log_int(rng, 8, 8192)
    if op == "ckpt":
        D = rng.choice([8, 16, 32, 64, 96, 128, 256, 512, 1024])
    H = _log_int(rng, 1, 40) if D <= 256 else 1
    T = _log_int(rng, 1, 32768)
    B = _log_int(rng, 1, 16)
    while B * H * T * D > 1 << 26 and B * H > 1:
        B, H = (max(1, B // 2), H) if B >= H else (B, max(1, H // 2))
    while B * H * T * D > 1 << 26:
        T = (T + 1) // 2
    ckpt = op == "norm_bwd" and D % 32 == 0 and rng.random() < 0.4
    return {k: v for k, v in _norm("", op, B, H, T, D, dtype, ckpt).items() if k != "name"}


# ---------------------------------------------------------------------------- inputs
def _lengths(c):
    """The lengths of a padded batch, before they are shuffled: 0 and T among them."""
    B, T = c["B"], c["T"]
    return [T] if B == 1 else [T * b // (B - 1) for b in range(B)]


def _rand(gen, *shape):
    return torch.randn(shape, generator=gen, device=DEV)


def _unit(x):
    return x / x.square().sum(-1, keepdim=True).sqrt()


def _pack(x):
    """The 8-bit form of activations: (codes uint8, scale bytes).  A group of G = min(D, 32) channels has
    the smallest power of two 2^e with amax / 2^e <= 448 (e >= -127), stored as e + 127."""
    D = x.shape[-1]
    G = min(D, 32)
    y = x.float().reshape(*x.shape[:-1], D // G, G)
    m, p = torch.frexp(y.abs().amax(-1, keepdim=True))                # amax = m 2^p, m in [1/2, 1)
    e = torch.where(m == 0, torch.full_like(p, -127), p - 9 + (m > 0.875).to(p.dtype)).clamp(min=-127)
    y = torch.ldexp(torch.ldexp(y, -(e // 2)), -(e - e // 2))
    codes = y.to(torch.float8_e4m3fn).view(torch.uint8).reshape(x.shape)
    return codes, (e + 127).to(torch.uint8).squeeze(-1)


def _unpack(codes, scales, dtype):
    D, n = codes.shape[-1], scales.shape[-1]
    y = codes.view(torch.float8_e4m3fn).float().reshape(*codes.shape[:-1], n, D // n)
    e = scales.to(torch.int32).unsqueeze(-1) - 127
    y = torch.ldexp(torch.ldexp(y, e // 2), e - e // 2)
    return y.reshape(codes.shape).to(dtype)


def prepare(case, seed):
    c = case
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    dt = DTYPES[c["dtype"]]
    B, H, T = c["B"], c["H"], c["T"]
    st = {"case": c}
    if c["op"].startswith("attn"):
        K, V = c["K"], c["V"]
        # slopes from 1/2 downwards over the heads, as fixed-decay layers set them
        slope = torch.exp2(-8.0 * torch.arange(1, H + 1, device=DEV) / H)
        st["g"] = -slope * (0.5 + 0.5 * torch.rand(H, generator=gen, device=DEV))
        S = 0.1 * _rand(gen, B, H, K, V)
        if c["op"] == "attn_step":
            st["q"], st["k"] = (_unit(_rand(gen, B, H, K)).to(dt) for _ in range(2))
            st["v"] = _rand(gen, B, H, V).to(dt)
            st["state"] = S
            return st
        st["q"], st["k"] = (_unit(_rand(gen, B, H, T, K)).to(dt) for _ in range(2))
        st["v"] = _rand(gen, B, H, T, V).to(dt)
        st["state_in"] = S
        st["lengths"] = None
        if c["ragged"]:
            lens = torch.tensor(_lengths(c), device=DEV, dtype=torch.int32)
            st["lengths"] = lens[torch.randperm(B, generator=gen, device=DEV)].contiguous()
        if c["op"] == "attn_fwd":
            st["out"] = torch.zeros(B, H, T, V, dtype=dt, device=DEV)      # rows behind a sequence stay as they are
        else:
            st["d_o"] = _rand(gen, B, H, T, V).to(dt)
            st["d_state"] = 0.1 * _rand(gen, B, H, K, V)
            if c["ckpt"]:
                for n in ("q", "k", "v"):
                    st[n] = _pack(st[n])
        return st
    D = c["D"]
    x = (0.5 + _rand(gen, B, H, T, D) * torch.exp(_rand(gen, B, H, T, 1) * 0.5)).to(dt)
    st["x"] = x
    if c["op"] == "ckpt":
        return st
    st["weight"] = 1.0 + 0.1 * _rand(gen, H, D)
    st["bias"] = 0.1 * _rand(gen, H, D)
    if c["op"] == "norm_bwd":
        xd = x.double()
        st["mean"] = xd.mean(-1).float()
        st["rstd"] = (xd.var(-1, unbiased=False) + EPS).rsqrt().float()
        st["dy"] = _rand(gen, B, H, T, D).to(dt)
        if c["ckpt"]:
            st["x"] = _pack(x)
    return st


# ---------------------------------------------------------------------------- plain forms
CHUNK = 128


def _valid(st, T):
    """(B, 1, T, 1) truth values of the tokens inside their sequence, and the (B, 1, 1, 1) lengths."""
    n = st["lengths"]
    if n is None:
        n = torch.full((st["case"]["B"],), T, device=DEV, dtype=torch.int32)
    n = n.view(-1, 1, 1, 1)
    return torch.arange(T, device=DEV).view(1, 1, T, 1) < n, n


def _kept(st, ok, x, other):
    """x at the tokens inside their sequence, `other` behind them."""
    return x if st["lengths"] is None else torch.where(ok, x, other)


def _chunks(x):
    B, H, T, D = x.shape
    N = -(-T // CHUNK)
    x = torch.nn.functional.pad(x, (0, 0, 0, N * CHUNK - T))
    return x.reshape(B, H, N, CHUNK, D)


def _pow(g, n):
    """exp(g n) for n >= 0, 0 for n < 0; the product in 64 bits (n reaches the sequence's length)."""
    return torch.where(n >= 0, torch.exp(g.double() * n.clamp(min=0)), 0.0).float()


def _tables(g, N):
    i = torch.arange(CHUNK, device=DEV)
    c = torch.arange(N, device=DEV)
    gh = g.view(1, -1, 1, 1, 1)
    inside = _pow(gh, (i.view(-1, 1) - i.view(1, -1)))                           # decay from token j to token i
    read = _pow(gh, (i + 1).view(-1, 1))                                         # chunk start to token i
    left = _pow(gh, (CHUNK - 1 - i).view(-1, 1))                                 # token i to chunk end
    across = _pow(g.view(1, -1, 1, 1), CHUNK * (c.view(-1, 1) - 1 - c.view(1, -1)))   # chunk end c' to chunk start c
    return inside, read, left, across


def _masked(st, T, *xs):
    ok, n = _valid(st, T)
    return [_kept(st, ok, x, 0.0) for x in xs], ok, n


def _states(k, v, left, across, g, S0):
    """The state at every chunk's start."""
    U = (k * left).transpose(-1, -2) @ v                                         # (B,H,N,K,V)
    B, H, N, K, V = U.shape
    S = (across @ U.reshape(B, H, N, K * V)).reshape(U.shape)
    first = _pow(g.view(1, -1, 1, 1, 1), (CHUNK * torch.arange(N, device=DEV)).view(N, 1, 1))
    return S + first * S0.unsqueeze(2)


def _plain_fwd(st):
    c, g = st["case"], st["g"]
    T, scale = c["T"], c["K"] ** -0.5
    (q, k, v), ok, n = _masked(st, T, st["q"].float(), st["k"].float(), st["v"].float())
    gh = g.view(1, -1, 1, 1)
    to_end = _pow(gh, n - 1 - torch.arange(T, device=DEV).view(1, 1, T, 1))
    state = (k * to_end).transpose(-1, -2) @ v + _pow(gh, n) * st["state_in"]
    qc, kc, vc = _chunks(q), _chunks(k), _chunks(v)
    inside, read, left, across = _tables(g, qc.shape[2])
    o = (qc @ kc.transpose(-1, -2) * inside) @ vc
    o += (qc * read) @ _states(kc, vc, left, across, g, st["state_in"])
    o = (scale * o).flatten(2, 3)[:, :, :T]
    return {"o": _kept(st, ok, o.to(st["q"].dtype), st["out"]), "state": state}


def _plain_bwd(st):
    c, g = st["case"], st["g"]
    T, scale = c["T"], c["K"] ** -0.5
    dt = st["d_o"].dtype
    q, k, v = (_unpack(*st[x], torch.float32) if c["ckpt"] else st[x].float() for x in ("q", "k", "v"))
    (q, k, v, d), ok, n = _masked(st, T, q, k, v, st["d_o"].float() * scale)
    gh = g.view(1, -1, 1, 1)
    at = torch.arange(T, device=DEV).view(1, 1, T, 1)
    to_end = _pow(gh, n - 1 - at) * ok
    dS = st["d_state"]
    d_in = (q * _pow(gh, at + 1)).transpose(-1, -2) @ d + _pow(gh, n) * dS
    qc, kc, vc, dc = _chunks(q), _chunks(k), _chunks(v), _chunks(d)
    inside, read, left, across = _tables(g, qc.shape[2])
    S = _states(kc, vc, left, across, g, st["state_in"])
    dvt = dc @ vc.transpose(-1, -2) * inside                                     # over (t, s)
    qkt = qc @ kc.transpose(-1, -2) * inside
    U = (qc * read).transpose(-1, -2) @ dc
    R = (across.transpose(-1, -2) @ U.flatten(3)).reshape(U.shape)               # dL/dS at every chunk's end
    dq = (dvt @ kc + (dc * read) @ S.transpose(-1, -2)).flatten(2, 3)[:, :, :T]
    dk = (dvt.transpose(-1, -2) @ qc + (vc * left) @ R.transpose(-1, -2)).flatten(2, 3)[:, :, :T]
    dv = (qkt.transpose(-1, -2) @ dc + (kc * left) @ R).flatten(2, 3)[:, :, :T]
    dk = dk + (v * to_end) @ dS.transpose(-1, -2)
    dv = dv + (k * to_end) @ dS
    dq, dk, dv = (_kept(st, ok, x, 0.0).to(dt) for x in (dq, dk, dv))
    return {"dq": dq, "dk": dk, "dv": dv, "dstate_in": d_in}


def _plain_step(st):
    q, k, v = (st[n].float() for n in ("q", "k", "v"))
    st["state"].mul_(torch.exp(st["g"]).view(1, -1, 1, 1)).add_(k.unsqueeze(-1) * v.unsqueeze(-2))
    o = (q.unsqueeze(-1) * st["state"]).sum(-2) * (q.shape[-1] ** -0.5)
    return {"o": o.to(st["q"].dtype), "state": st["state"]}


def _plain_norm(st):
    x = st["x"].float()
    mean = x.mean(-1, keepdim=True)
    xc = x - mean
    rstd = (xc.square().mean(-1, keepdim=True) + EPS).rsqrt()
    y = xc * rstd * st["weight"].unsqueeze(1) + st["bias"].unsqueeze(1)
    return {"y": y.to(st["x"].dtype), "mean": mean.squeeze(-1), "rstd": rstd.squeeze(-1)}


def _plain_norm_bwd(st):
    dy = st["dy"].float()
    x = _unpack(*st["x"], torch.float32) if st["case"]["ckpt"] else st["x"].float()
    rstd = st["rstd"].unsqueeze(-1)
    xh = (x - st["mean"].unsqueeze(-1)) * rstd
    wdy = dy * st["weight"].unsqueeze(1)
    dx = rstd * (wdy - wdy.mean(-1, keepdim=True) - xh * (wdy * xh).mean(-1, keepdim=True))
    return {"dx": dx.to(st["dy"].dtype), "dweight": (dy * xh).sum((0, 2)), "dbias": dy.sum((0, 2))}


def _plain_ckpt(st):
    codes, scales = _pack(st["x"])
    return {"scales": scales, "values": _unpack(codes, scales, st["x"].dtype)}


_PLAIN = {"attn_fwd": _plain_fwd, "attn_bwd": _plain_bwd, "attn_step": _plain_step, "norm_fwd": _plain_norm,
          "norm_bwd": _plain_norm_bwd, "ckpt": _plain_ckpt}


# ---------------------------------------------------------------------------- the framework's calls
def _own(st):
    import gated_delta_rule_47_amd as kda
    op = st["case"]["op"]
    if op == "attn_fwd":
        o, state = kda.decay_attn_fwd(st["q"], st["k"], st["v"], st["g"], st["state_in"], lengths=st["lengths"],
                                      out=st["out"])
        return {"o": o, "state": state}
    if op == "attn_step":
        o = kda.decay_attn_step(st["q"], st["k"], st["v"], st["g"], st["state"])
        return {"o": o, "state": st["state"]}
    if op == "attn_bwd":
        return kda.decay_attn_bwd(st["q"], st["k"], st["v"], st["g"], st["state_in"], st["d_o"], st["d_state"],
                                  lengths=st["lengths"])
    if op == "norm_fwd":
        y, mean, rstd = kda.layer_norm_fwd(st["x"], st["weight"], st["bias"], eps=EPS)
        return {"y": y, "mean": mean, "rstd": rstd}
    if op == "norm_bwd":
        dx, dw, db = kda.layer_norm_bwd(st["x"], st["weight"], st["mean"], st["rstd"], st["dy"])
        return {"dx": dx, "dweight": dw, "dbias": db}
    codes, scales = kda.ckpt_pack(st["x"])
    return {"scales": scales, "values": kda.ckpt_unpack(codes, scales, st["x"].dtype)}


def run(state):
    if own:
        return _own(state)
    return _PLAIN[state["case"]["op"]](state)


# ---------------------------------------------------------------------------- what a pass cannot do without
def work(case):
    c = case
    es = 2 if c["dtype"] == "bf16" else 4
    if c["op"].startswith("attn"):
        B, H, K, V = c["B"], c["H"], c["K"], c["V"]
        n = H * (sum(_lengths(c)) if c["ragged"] else B * c["T"])                # head-tokens
        state = B * H * K * V * 4
        if c["op"] == "attn_bwd":
            ins = (2 * K + V) + (2 * K / min(K, 32) + V / min(V, 32)) if c["ckpt"] else (2 * K + V) * es
            return {"bytes": n * (ins + V * es + (2 * K + V) * es) + 3 * state, "flops": 10 * n * K * V}
        return {"bytes": n * 2 * (K + V) * es + 2 * state, "flops": 4 * n * K * V}
    D, rows = c["D"], c["B"] * c["H"] * c["T"]
    n = rows * D
    par = c["H"] * D * 4
    if c["op"] == "norm_fwd":
        return {"bytes": 2 * n * es + 8 * rows + 2 * par, "flops": 8 * n}
    if c["op"] == "norm_bwd":
        return {"bytes": n * (2 * es + (1 + 1 / min(D, 32) if c["ckpt"] else es)) + 8 * rows + 3 * par,
                "flops": 14 * n}
    # stored once, read back once
    return {"bytes": 2 * n * es + 2 * n * (1 + 1 / min(D, 32)), "flops": 4 * n}


# ---------------------------------------------------------------------------- the definition in 64 bits
def _exact_value(codes, scales):
    """e4m3 by its definition: sign, 4 bits of exponent (bias 7), 3 of mantissa, times 2^(scale byte - 127)."""
    b = codes.to(torch.int64)
    exp, man = (b >> 3) & 15, (b & 7).double()
    mag = torch.where(exp == 0, man * 2.0 ** -9, (8 + man) * torch.exp2((exp - 10).double()))
    mag = torch.where(b >= 128, -mag, mag)
    G = codes.shape[-1] // scales.shape[-1]
    return mag * torch.exp2(scales.double() - 127).repeat_interleave(G, -1)


def _exact_ckpt(st):
    x = st["x"].double()
    D = x.shape[-1]
    G = min(D, 32)
    y = x.reshape(*x.shape[:-1], D // G, G)
    amax = y.abs().amax(-1, keepdim=True)
    e = torch.ceil(torch.log2((amax / 448).clamp(min=2.0 ** -127)))
    e = torch.where(amax > 448 * torch.exp2(e), e + 1, torch.where(amax <= 448 * torch.exp2(e - 1), e - 1, e))
    e = e.clamp(min=-127)
    y = y / torch.exp2(e)
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    return {"scales": None, "values": (torch.round(y / step) * step * torch.exp2(e)).reshape(x.shape)}


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op in ("attn_fwd", "attn_bwd"):
        # token by token: forward for the read (or dq), backward for the other gradients
        ok, _ = _valid(st, case["T"])
        x = {n: _exact_value(*st[n]) if isinstance(st[n], tuple) else st[n].double() for n in ("q", "k", "v")}
        q, k, v = (torch.where(ok, x[n], 0.0) for n in ("q", "k", "v"))
        a = torch.exp(st["g"].double()).view(1, -1, 1, 1)
        S, scale = st["state_in"].double(), case["K"] ** -0.5
        if op == "attn_fwd":
            o = torch.empty_like(v)
            for t in range(case["T"]):
                S = S * torch.where(ok[:, :, t, None], a, 1.0) + k[:, :, t, :, None] * v[:, :, t, None, :]
                o[:, :, t] = (q[:, :, t, None, :] @ S).squeeze(-2)
            return {"o": torch.where(ok, o * scale, st["out"].double()), "state": S}
        d = torch.where(ok, st["d_o"].double() * scale, 0.0)
        R = st["d_state"].double()
        dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
        for t in range(case["T"]):
            S = S * torch.where(ok[:, :, t, None], a, 1.0) + k[:, :, t, :, None] * v[:, :, t, None, :]
            dq[:, :, t] = (S @ d[:, :, t, :, None]).squeeze(-1)
        for t in reversed(range(case["T"])):
            R = R + q[:, :, t, :, None] * d[:, :, t, None, :]
            dk[:, :, t] = (R @ v[:, :, t, :, None]).squeeze(-1)
            dv[:, :, t] = (k[:, :, t, None, :] @ R).squeeze(-2)
            R = R * torch.where(ok[:, :, t, None], a, 1.0)
        return {"dq": dq * ok, "dk": dk * ok, "dv": dv * ok, "dstate_in": R}
    if op == "attn_step":
        S = st["state"].double() * torch.exp(st["g"].double()).view(1, -1, 1, 1)
        S = S + st["k"].double().unsqueeze(-1) * st["v"].double().unsqueeze(-2)
        o = torch.einsum("bhk,bhkv->bhv", st["q"].double(), S) * case["K"] ** -0.5
        return {"o": o, "state": S}
    if op == "ckpt":
        return _exact_ckpt(st)
    w, b = st["weight"].double()[:, None], st["bias"].double()[:, None]
    if op == "norm_fwd":
        x = st["x"].double()
        var, mean = torch.var_mean(x, -1, unbiased=False, keepdim=True)
        rstd = 1 / torch.sqrt(var + EPS)
        return {"y": (x - mean) * rstd * w + b, "mean": mean.squeeze(-1), "rstd": rstd.squeeze(-1)}
    x = _exact_value(*st["x"]) if case["ckpt"] else st["x"].double()
    dy, r = st["dy"].double(), st["rstd"].double().unsqueeze(-1)
    xh = (x - st["mean"].double().unsqueeze(-1)) * r
    dxh = dy * w
    D = x.shape[-1]
    dx = r / D * (D * dxh - dxh.sum(-1, keepdim=True) - xh * (dxh * xh).sum(-1, keepdim=True))
    return {"dx": dx, "dweight": (dy * xh).sum(2).sum(0), "dbias": dy.sum(2).sum(0)}
