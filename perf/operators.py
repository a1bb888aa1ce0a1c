"""Measured cases of the short causal convolution, the selective state space scan (prompts and
single tokens of both) and the copies between state slots.

``run`` makes either the plain form of an operator (elementary torch operations in 32 bits) or,
where ``own`` is true, the call a user makes of ``gated_delta_rule_wise_gb300``.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


# ---------------------------------------------------------------- cases

def _conv(name, B, H, T, d, W, dtype, silu=True, bias=False, state=False, ragged=False,
          token_major=True):
    return dict(name=name, op="conv", B=B, H=H, T=T, d=d, W=W, dtype=dtype, silu=silu, bias=bias,
                state=state, ragged=ragged, token_major=token_major)


def _conv_step(name, N, H, d, W, dtype, silu=True, bias=False, slots=True):
    return dict(name=name, op="conv_step", N=N, H=H, d=d, W=W, dtype=dtype, silu=silu, bias=bias,
                slots=slots)


def _scan(name, B, T, D, N, G, dtype, gate=True, state=False, ragged=False, softplus=True):
    return dict(name=name, op="scan", B=B, T=T, D=D, N=N, G=G, dtype=dtype, gate=gate, state=state,
                ragged=ragged, softplus=softplus)


def _step(name, R, D, N, G, dtype, gate=True, slots=True, softplus=True):
    return dict(name=name, op="step", R=R, D=D, N=N, G=G, dtype=dtype, gate=gate, slots=slots,
                softplus=softplus)


def _copy(name, L, P, page, n, dtype, fork=1):
    return dict(name=name, op="copy", L=L, P=P, page=page, n=n, dtype=dtype, fork=fork)


def listed():
    return [
        # the queries of one long prompt, 32 heads of 128 channels as the projection wrote them
        # (token by token), on their way to the chunked prefill
        _conv("conv prompt 32x32768x128", 1, 32, 32768, 128, 4, "bf16"),
        # a padded batch of prompts continued from a state, with a bias and a channel count that
        # no vector divides
        _conv("conv padded batch odd f32", 5, 1, 1000, 2050, 4, "f32", bias=True, state=True,
              ragged=True),
        # one token of 256 sequences, 32 heads of 128 channels, states in a pool
        _conv_step("conv step 256x32x128", 256, 32, 128, 4, "bf16"),
        # one token of one sequence: latency
        _conv_step("conv step 1x1x1536", 1, 1, 1536, 4, "bf16", bias=True, slots=False),
        # one long prompt: few channels, many tokens
        _scan("scan prompt 16384x4096", 1, 16384, 4096, 16, 1, "bf16"),
        # a padded batch of ordinary prompts that continue from states
        _scan("scan padded batch 16x1000x2048", 16, 1000, 2048, 16, 1, "bf16", state=True,
              ragged=True),
        # a short prompt: latency
        _scan("scan prompt 128x1536", 1, 128, 1536, 16, 1, "bf16"),
        # float32, groups, an odd length, no gate, the step sizes given as they are
        _scan("scan groups f32 3x777x1000", 3, 777, 1000, 64, 4, "f32", gate=False,
              softplus=False),
        # one token of 256 sequences, states in a pool
        _step("scan step 256x4096", 256, 4096, 16, 1, "bf16"),
        # one token of one sequence: latency
        _step("scan step 1x1536", 1, 1536, 16, 1, "bf16", slots=False),
        # compaction of the delta rule's float32 states, 32 x 128 x 128 each: 48 sequences move
        # to the slots of ended ones
        _copy("copy 48 states of 2 MiB", 1, 160, 32 * 128 * 128, 48, "f32"),
        # one sequence's convolution states in 24 layers forked to four samples
        _copy("fork conv states 24 layers", 24, 64, 3 * 4096, 4, "bf16", fork=4),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["conv", "conv_step", "scan", "scan", "step", "copy"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    wide = 2 if dtype == "f32" else 1
    yes = lambda p=0.5: rng.random() < p  # noqa: E731
    if op == "conv":
        B, H, d = _log_int(rng, 1, 8), _log_int(rng, 1, 32), _log_int(rng, 16, 256)
        if yes(0.3):
            H, d = 1, _log_int(rng, 256, 8192)
        if yes():
            d = -(-d // 8) * 8
        T = max(1, min(_log_int(rng, 1, 32768), 32 * 32768 * 128 // (wide * B * H * d)))
        c = _conv("", B, H, T, d, rng.choice([2, 3, 4, 4]), dtype, yes(0.8), yes(), yes(),
                  yes(0.4), yes(0.7))
    elif op == "conv_step":
        H, d = _log_int(rng, 1, 32), _log_int(rng, 16, 256)
        if yes(0.3):
            H, d = 1, _log_int(rng, 256, 4096)
        if yes():
            d = -(-d // 8) * 8
        N = max(1, min(_log_int(rng, 1, 512), 256 * 32 * 128 // (wide * H * d)))
        c = _conv_step("", N, H, d, rng.choice([2, 3, 4, 4]), dtype, yes(0.8), yes(), yes(0.7))
    elif op == "scan":
        G = rng.choice([1, 1, 1, 2, 4])
        D = max(1, _log_int(rng, 16, 8192) // G) * G
        if yes():
            D = -(-D // (8 * G)) * 8 * G
        N = rng.choice([8, 16, 16, 16, 32, 64])
        B = _log_int(rng, 1, 16)
        T = max(1, min(_log_int(rng, 1, 16384), 16000 * 4096 * 16 // (wide * B * D * max(N, 16))))
        c = _scan("", B, T, D, N, G, dtype, yes(0.7), yes(), yes(0.4), yes(0.8))
    elif op == "step":
        G = rng.choice([1, 1, 1, 2, 4])
        D = max(1, _log_int(rng, 16, 8192) // G) * G
        if yes():
            D = -(-D // (8 * G)) * 8 * G
        N = rng.choice([8, 16, 16, 16, 32, 64])
        R = max(1, min(_log_int(rng, 1, 512), 256 * 4096 * 16 // (D * max(N, 16))))
        c = _step("", R, D, N, G, dtype, yes(0.7), yes(0.7), yes(0.8))
    else:
        page = _log_int(rng, 100, 32 * 128 * 128)
        if yes():
            page = -(-page // 16) * 16
        L = _log_int(rng, 1, 48)
        room = 48 * 32 * 128 * 128 // (L * page)
        fork = rng.choice([1, 1, 2, 8])
        n = max(1, min(_log_int(rng, 1, 256), room) // fork) * fork
        P = 2 * n + rng.randrange(1, 17)
        if L * page * n > 48 * 32 * 128 * 128:
            L, n, P = 1, fork, 3 * fork
        c = _copy("", L, P, page, n, dtype, fork)
    del c["name"]
    return c


# ---------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _normal(g, shape, sd=1.0, dtype=torch.float32):
    return torch.randn(shape, generator=g, device=DEV).mul_(sd).to(dtype)


def _lengths(g, B, T):
    """Lengths of a padded batch: anywhere in it, the first one full."""
    n = torch.randint(0, T + 1, (B,), generator=g, device=DEV, dtype=torch.int32)
    n[0] = T
    return n


def _slots(g, N, P):
    return torch.randperm(P, generator=g, device=DEV)[:N].to(torch.int32)


def _scan_inputs(g, lead, D, N, G, dt, gate, softplus):
    """u, delta, B, C, z of a block: B and C are slices of one projection, z of another, as the
    block's matrix products leave them; step sizes exp(U(log 1e-3, log 0.1)) around their bias."""
    s = {"A": -(torch.arange(1, N + 1, device=DEV, dtype=torch.float32)
                * torch.exp(0.1 * _normal(g, (D, N))))}
    s["u"] = _normal(g, lead + (D,), 1.0, dt)
    step = torch.exp(torch.rand(D, generator=g, device=DEV) * math.log(100.0) + math.log(1e-3))
    if softplus:
        s["delta"] = _normal(g, lead + (D,), 0.5, dt)
        s["delta_bias"] = step + torch.log(-torch.expm1(-step))
    else:
        s["delta"] = (step * torch.exp(_normal(g, lead + (D,), 0.3))).to(dt)
        s["delta_bias"] = None
    rank = 8 * max(1, D // 128)
    proj = _normal(g, lead + (rank + 2 * G * N,), 1.0, dt)
    s["B"] = proj[..., rank:rank + G * N].unflatten(-1, (G, N))
    s["C"] = proj[..., rank + G * N:].unflatten(-1, (G, N))
    s["z"] = _normal(g, lead + (2 * D,), 1.0, dt)[..., D:] if gate else None
    s["Dskip"] = 1.0 + 0.1 * _normal(g, (D,))
    return s


def prepare(case, seed):
    g, c, dt = _gen(seed), case, TYPES[case["dtype"]]
    s = {"op": c["op"]}
    if c["op"] == "conv":
        B, H, T, d, W = (c[k] for k in "BHTdW")
        x = _normal(g, (B, T, H, d) if c["token_major"] else (B, H, T, d), 1.0, dt)
        s["x"] = x.transpose(1, 2) if c["token_major"] else x
        s["w"] = _normal(g, (H, d, W), 0.5)
        s["bias"] = _normal(g, (H, d), 0.2) if c["bias"] else None
        s["s0"] = _normal(g, (B, H, W - 1, d), 1.0, dt) if c["state"] else None
        s["lens"] = _lengths(g, B, T) if c["ragged"] else None
        s["silu"] = c["silu"]
        s["y"] = torch.zeros((B, H, T, d), dtype=dt, device=DEV)
    elif c["op"] == "conv_step":
        N, H, d, W = (c[k] for k in "NHdW")
        P = N + N // 4 + 1 if c["slots"] else N
        s["x"] = _normal(g, (N, H, d), 1.0, dt)
        s["w"] = _normal(g, (H, d, W), 0.5)
        s["bias"] = _normal(g, (H, d), 0.2) if c["bias"] else None
        s["S"] = _normal(g, (P, H, W - 1, d), 1.0, dt)
        s["slots"] = _slots(g, N, P) if c["slots"] else None
        s["silu"] = c["silu"]
    elif c["op"] == "scan":
        B, T, D, N, G = (c[k] for k in "BTDNG")
        s.update(_scan_inputs(g, (B, T), D, N, G, dt, c["gate"], c["softplus"]))
        s["h0"] = _normal(g, (B, D, N), 0.5) if c["state"] else None
        s["lens"] = _lengths(g, B, T) if c["ragged"] else None
        s["softplus"] = c["softplus"]
        s["y"] = torch.zeros((B, T, D), dtype=dt, device=DEV)
    elif c["op"] == "step":
        R, D, N, G = (c[k] for k in "RDNG")
        P = R + R // 4 + 1 if c["slots"] else R
        s.update(_scan_inputs(g, (R,), D, N, G, dt, c["gate"], c["softplus"]))
        s["S"] = _normal(g, (P, D, N), 0.5)
        s["slots"] = _slots(g, R, P) if c["slots"] else None
        s["softplus"] = c["softplus"]
    else:
        L, P, page, n = (c[k] for k in ("L", "P", "page", "n"))
        s["pool"] = _normal(g, (L, P, page), 1.0, dt)
        order = torch.randperm(P, generator=g, device=DEV).to(torch.int32).cpu()
        k = n // c["fork"]  # sources, each copied to `fork` free slots
        s["src"] = order[:k].repeat_interleave(c["fork"]).contiguous()
        s["dst"] = order[k:k + n].contiguous()
    return s


# ---------------------------------------------------------------- plain forms

def _silu(x):
    return x / (1.0 + torch.exp(-x))


def _softplus(x):
    return torch.clamp(x, min=0.0) + torch.log1p(torch.exp(-torch.abs(x)))


def _taps(full, w, T):
    """sum_j w[..., j] full[:, :, j:j+T] with full [B,H,W-1+T,d], w [H,d,W]."""
    return sum(full[:, :, j:j + T] * w[:, None, :, j] for j in range(w.shape[-1]))


def _plain_conv(s):
    x, w, dt = s["x"], s["w"], s["x"].dtype
    B, H, T, d = x.shape
    W = w.shape[-1]
    past = s["s0"] if s["s0"] is not None else x.new_zeros((B, H, W - 1, d))
    full = torch.cat([past, x], 2).float()
    y = _taps(full, w, T)
    if s["bias"] is not None:
        y = y + s["bias"][:, None, :]
    if s["silu"]:
        y = _silu(y)
    if s["lens"] is None:
        s["y"].copy_(y)
        return s["y"], full[:, :, T:].to(dt)
    live = torch.arange(T, device=DEV)[None] < s["lens"][:, None]
    s["y"].copy_(torch.where(live[:, None, :, None], y.to(dt), s["y"]))
    at = s["lens"].long()[:, None] + torch.arange(W - 1, device=DEV)
    last = full.transpose(1, 2)[torch.arange(B, device=DEV)[:, None], at]
    return s["y"], last.transpose(1, 2).to(dt).contiguous()


def _plain_conv_step(s):
    x, w, S, dt = s["x"], s["w"], s["S"], s["x"].dtype
    old = S if s["slots"] is None else S[s["slots"].long()]
    full = torch.cat([old, x[:, :, None]], 2)
    y = _taps(full.float(), w, 1)[:, :, 0]
    if s["bias"] is not None:
        y = y + s["bias"]
    if s["silu"]:
        y = _silu(y)
    if s["slots"] is None:
        S.copy_(full[:, :, 1:])
    else:
        S[s["slots"].long()] = full[:, :, 1:]
    return y.to(dt), S


def _channels(x, D):
    """[..., G, N] per group to [..., D, N] per channel."""
    return x.float().repeat_interleave(D // x.shape[-2], -2)


def _plain_scan(s):
    u, dt = s["u"], s["u"].dtype
    B, T, D = u.shape
    step = s["delta"].float()
    if s["delta_bias"] is not None:
        step = step + s["delta_bias"]
    if s["softplus"]:
        step = _softplus(step)
    live = None
    if s["lens"] is not None:  # beyond its length a row neither decays nor adds
        live = (torch.arange(T, device=DEV)[None] < s["lens"][:, None])[..., None]
        step = torch.where(live, step, 0.0)
    a = torch.exp(step[..., None] * s["A"])
    h = (step * u.float())[..., None] * _channels(s["B"], D)
    if s["h0"] is not None:
        h[:, 0] += a[:, 0] * s["h0"]
    reach = 1
    while reach < T:  # pairs (a, h) joined over spans that double
        h[:, reach:] += a[:, reach:] * h[:, :-reach].clone()
        a[:, reach:] *= a[:, :-reach].clone()
        reach *= 2
    y = (h * _channels(s["C"], D)).sum(-1) + s["Dskip"] * u.float()
    if s["z"] is not None:
        y = y * _silu(s["z"].float())
    y = y.to(dt)
    s["y"].copy_(y if live is None else torch.where(live, y, s["y"]))
    return s["y"], h[:, -1].clone()


def _plain_step(s):
    u, S, dt = s["u"], s["S"], s["u"].dtype
    step = s["delta"].float()
    if s["delta_bias"] is not None:
        step = step + s["delta_bias"]
    if s["softplus"]:
        step = _softplus(step)
    old = S if s["slots"] is None else S[s["slots"].long()]
    D = u.shape[-1]
    h = torch.exp(step[..., None] * s["A"]) * old \
        + (step * u.float())[..., None] * _channels(s["B"], D)
    y = (h * _channels(s["C"], D)).sum(-1) + s["Dskip"] * u.float()
    if s["z"] is not None:
        y = y * _silu(s["z"].float())
    if s["slots"] is None:
        S.copy_(h)
    else:
        S[s["slots"].long()] = h
    return y.to(dt), S


def _plain_copy(s):
    src, dst = s["src"].to(DEV).long(), s["dst"].to(DEV).long()
    s["pool"][:, dst] = s["pool"][:, src]
    return s["pool"]


PLAIN = {"conv": _plain_conv, "conv_step": _plain_conv_step, "scan": _plain_scan,
         "step": _plain_step, "copy": _plain_copy}


def run(s):
    if not own:
        return PLAIN[s["op"]](s)
    import gated_delta_rule_wise_gb300 as kda
    if s["op"] == "conv":
        return kda.short_conv(s["x"], s["w"], bias=s["bias"], s0=s["s0"], lens=s["lens"],
                              act=kda.KDA_ACT_SILU if s["silu"] else kda.KDA_ACT_NONE, out=s["y"])
    if s["op"] == "conv_step":
        y = kda.short_conv_step(s["x"], s["w"], s["S"], bias=s["bias"], slots=s["slots"],
                                act=kda.KDA_ACT_SILU if s["silu"] else kda.KDA_ACT_NONE)
        return y, s["S"]
    if s["op"] == "scan":
        return kda.selective_scan(s["u"], s["delta"], s["A"], s["B"], s["C"], D=s["Dskip"],
                                  z=s["z"], delta_bias=s["delta_bias"], h0=s["h0"],
                                  lens=s["lens"], softplus=s["softplus"], out=s["y"])
    if s["op"] == "step":
        y = kda.selective_step(s["u"], s["delta"], s["A"], s["B"], s["C"], s["S"], D=s["Dskip"],
                               z=s["z"], delta_bias=s["delta_bias"], slots=s["slots"],
                               softplus=s["softplus"])
        return y, s["S"]
    kda.state_copy(s["pool"], s["src"], s["dst"], layered=True)
    return s["pool"]


# ---------------------------------------------------------------- what a pass cannot do without

def _tokens(c):
    """Tokens of a batch; of a padded one the first row and on average half of each other."""
    return c["T"] * ((c["B"] + 1) / 2 if c["ragged"] else c["B"])


def work(case):
    c = case
    e = 4 if c["dtype"] == "f32" else 2
    if c["op"] == "conv":
        n = _tokens(c) * c["H"] * c["d"]
        row = c["B"] * c["H"] * (c["W"] - 1) * c["d"] * e
        return {"bytes": 2 * n * e + row * (2 if c["state"] else 1)
                + c["H"] * c["d"] * 4 * (c["W"] + c["bias"]),
                "flops": n * (2 * c["W"] + 4 * c["silu"])}
    if c["op"] == "conv_step":
        n = c["N"] * c["H"] * c["d"]
        return {"bytes": 2 * n * e + 2 * (c["W"] - 1) * n * e
                + c["H"] * c["d"] * 4 * (c["W"] + c["bias"]),
                "flops": n * (2 * c["W"] + 4 * c["silu"])}
    if c["op"] == "scan":
        n, h = _tokens(c) * c["D"], c["B"] * c["D"] * c["N"]
        return {"bytes": n * e * (4 if c["gate"] else 3) + 2 * _tokens(c) * c["G"] * c["N"] * e
                + 4 * h * (2 if c["state"] else 1) + 4 * c["D"] * (c["N"] + 2),
                "flops": n * c["N"] * 7 + n * 8}
    if c["op"] == "step":
        n, h = c["R"] * c["D"], c["R"] * c["D"] * c["N"]
        return {"bytes": 8 * h + n * e * (4 if c["gate"] else 3) + 2 * c["R"] * c["G"] * c["N"] * e
                + 4 * c["D"] * (c["N"] + 2), "flops": 7 * h + 8 * n}
    k = c["n"] // c["fork"]
    return {"bytes": c["L"] * c["page"] * e * (c["n"] + k), "flops": 0}


# ---------------------------------------------------------------- 64 bits

def _d(x):
    return None if x is None else x.to(torch.float64)


def _exact_act(y, silu):
    return y * torch.sigmoid(y) if silu else y


def _exact_conv(s):
    """Token by token from the definition, one sequence at a time: a window that shifts."""
    x, w, bias = _d(s["x"]), _d(s["w"]), _d(s["bias"])
    B, H, T, d = x.shape
    W = w.shape[-1]
    y, last = _d(s["y"]).clone(), []
    for b in range(B):
        n = T if s["lens"] is None else int(s["lens"][b])
        past = torch.zeros((H, W - 1, d), dtype=torch.float64, device=DEV) \
            if s["s0"] is None else _d(s["s0"][b])
        line = torch.cat([past, x[b, :, :n]], 1)
        if n:
            win = line.unfold(1, W, 1)  # [H, n, d, W]
            v = torch.einsum("hndw,hdw->hnd", win, w)
            y[b, :, :n] = _exact_act(v if bias is None else v + bias[:, None], s["silu"])
        last.append(line[:, line.shape[1] - (W - 1):])
    return y, torch.stack(last)


def _exact_conv_step(s):
    S, x, w, bias = _d(s["S"]).clone(), _d(s["x"]), _d(s["w"]), _d(s["bias"])
    rows = torch.arange(x.shape[0], device=DEV) if s["slots"] is None else s["slots"].long()
    line = torch.cat([S[rows], x.unsqueeze(2)], 2)  # [N, H, W, d]
    v = torch.einsum("nhwd,hdw->nhd", line, w)
    S[rows] = line[:, :, 1:]
    return _exact_act(v if bias is None else v + bias, s["silu"]), S


def _exact_token(h, A, u, delta, Bm, Cm, bias, Dskip, z, softplus):
    """One token for rows [R]: h [R, D, N] in, (y, h) out."""
    R, D = u.shape
    dt = delta if bias is None else delta + bias
    if softplus:
        dt = torch.logaddexp(dt, torch.zeros_like(dt))
    g = torch.arange(D, device=DEV) // (D // Bm.shape[1])
    h = torch.exp(dt.unsqueeze(-1) * A) * h + (dt * u).unsqueeze(-1) * Bm[:, g]
    y = torch.einsum("rdn,rdn->rd", h, Cm[:, g]) + Dskip * u
    return (y if z is None else y * z * torch.sigmoid(z)), h


def _exact_scan(s):
    B, T, D = s["u"].shape
    A, bias, Dskip = _d(s["A"]), _d(s["delta_bias"]), _d(s["Dskip"])
    h = _d(s["h0"]) if s["h0"] is not None else torch.zeros((B,) + A.shape, dtype=torch.float64,
                                                            device=DEV)
    y = _d(s["y"]).clone()
    for t in range(T):
        z = None if s["z"] is None else _d(s["z"][:, t])
        v, new = _exact_token(h, A, _d(s["u"][:, t]), _d(s["delta"][:, t]), _d(s["B"][:, t]),
                              _d(s["C"][:, t]), bias, Dskip, z, s["softplus"])
        if s["lens"] is None:
            y[:, t], h = v, new
        else:
            live = (s["lens"] > t)[:, None]
            y[:, t] = torch.where(live, v, y[:, t])
            h = torch.where(live[..., None], new, h)
    return y, h


def _exact_step(s):
    S = _d(s["S"]).clone()
    rows = torch.arange(s["u"].shape[0], device=DEV) if s["slots"] is None else s["slots"].long()
    y, S[rows] = _exact_token(S[rows], _d(s["A"]), _d(s["u"]), _d(s["delta"]), _d(s["B"]),
                              _d(s["C"]), _d(s["delta_bias"]), _d(s["Dskip"]), _d(s["z"]),
                              s["softplus"])
    return y, S


def _exact_copy(s):
    pool = _d(s["pool"])
    for i, j in zip(s["src"].tolist(), s["dst"].tolist()):
        pool[:, j] = pool[:, i]
    return pool


EXACT = {"conv": _exact_conv, "conv_step": _exact_conv_step, "scan": _exact_scan,
         "step": _exact_step, "copy": _exact_copy}


def exact(case, seed):
    return EXACT[case["op"]](prepare(case, seed))
