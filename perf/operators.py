"""Linear attention with a decay for each head (whole sequences, their gradient, single
tokens) and the group norm with gate or activation that follows it: cases, inputs, the
operators in plain torch operations, and their values in 64 bits.

  linear attention   S_t = lam_h S_{t-1} + k_t (x) v_t,  o_t = scale q_t . S_t,  lam_h = exp(log_decay[h])
  group norm         y = act((x - mean) rstd w + b) [silu(z)], statistics over positions and a group's channels
"""
import math

import torch

own = False

DEV = "cuda"
CHUNK = 128
EPS = 1e-5
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # a short prompt, one chunk and a piece of another: what a request costs at the least
        dict(name="fwd_short", op="fwd", B=1, L=77, H=8, G=8, K=64, V=64, io="bf16", ragged=False, h0=False),
        # one prompt that continues a conversation (a state is carried in)
        dict(name="fwd_prompt", op="fwd", B=1, L=4096, H=16, G=16, K=128, V=128, io="bf16", ragged=False, h0=True),
        # a batch of long documents; three heads share each group of queries and keys
        dict(name="fwd_long", op="fwd", B=4, L=8000, H=24, G=8, K=128, V=64, io="bf16", ragged=False, h0=False),
        # a padded batch of requests in 32 bits
        dict(name="fwd_ragged_f32", op="fwd", B=8, L=1000, H=8, G=8, K=64, V=64, io="f32", ragged=True, h0=True),
        # a training step's sequences
        dict(name="bwd_train", op="bwd", B=4, L=4096, H=16, G=16, K=128, V=128, io="bf16", ragged=False, h0=False),
        # a padded batch of odd length with shared queries and keys and a carried state
        dict(name="bwd_ragged_shared", op="bwd", B=4, L=2047, H=24, G=8, K=128, V=64, io="bf16", ragged=True, h0=True),
        # one user's next token
        dict(name="step_one", op="step", B=1, H=16, G=16, K=128, V=128, io="bf16", norm=False),
        # a serving batch's next tokens, with the norm and gate that follow
        dict(name="step_batch", op="step", B=64, H=24, G=24, K=128, V=64, io="bf16", norm=True),
        # the gated norm per head of a batch of single tokens
        dict(name="norm_tokens", op="norm", M=64, S=1, C=2048, groups=16, io="bf16", act="none", gate=True),
        # a convolutional block's norm and activation over a 64 x 64 grid
        dict(name="norm_grid", op="norm", M=16, S=4096, C=512, groups=32, io="bf16", act="silu", gate=False),
        # the gated norm's gradient over a training step's tokens
        dict(name="norm_bwd_tokens", op="norm_bwd", M=32768, S=1, C=1536, groups=24, io="bf16", act="none", gate=True),
        # the convolutional block's gradient: ten channels a group, an odd number of positions, 32 bits
        dict(name="norm_bwd_grid_f32", op="norm_bwd", M=8, S=1025, C=320, groups=32, io="f32", act="silu", gate=False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["fwd", "fwd", "bwd", "bwd", "step", "norm", "norm_bwd"])
    io = rng.choice(["bf16", "bf16", "f32"])
    if op in ("norm", "norm_bwd"):
        while True:
            tokens = rng.random() < 0.5
            groups, per = rng.randint(1, 32), _log_int(rng, 2, 40) * rng.choice([1, 2, 4])
            M = _log_int(rng, 1, 32768 if tokens else 32)
            S = 1 if tokens else _log_int(rng, 2, 9000)
            if M * S * groups * per <= 32768 * 1536:
                break
        gate = rng.random() < (0.8 if tokens else 0.1)
        return dict(op=op, M=M, S=S, C=groups * per, groups=groups, io=io,
                    act="none" if gate else rng.choice(["none", "silu"]), gate=gate)
    G = _log_int(rng, 1, 16)
    H = G * rng.choice([1, 1, 2, 3])
    K, V = rng.choice([64, 128]), rng.choice([64, 128])
    if op == "step":
        return dict(op=op, B=_log_int(rng, 1, 128), H=H, G=G, K=K, V=V, io=io, norm=rng.random() < 0.5)
    most = (4 * 8000 * 24 if op == "fwd" else 4 * 4096 * 16) // (1 if io == "bf16" else 2)
    while True:
        B, L = _log_int(rng, 1, 16), _log_int(rng, 1, 8192)
        if B * L * H * max(K, V) <= most * 64:
            break
    return dict(op=op, B=B, L=L, H=H, G=G, K=K, V=V, io=io, ragged=rng.random() < 0.4, h0=rng.random() < 0.5)


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    c = dict(case)
    io = TYPES[c["io"]]

    def normal(*shape, dtype=io, scale=1.0):
        return (torch.randn(shape, generator=g, device=DEV) * scale).to(dtype)

    s = {"case": c}
    if c["op"] in ("norm", "norm_bwd"):
        M, S, C, G = c["M"], c["S"], c["C"], c["groups"]
        # groups of different spread and offset, as activations have
        spread = torch.exp(torch.randn((1, 1, G, 1), generator=g, device=DEV) * 0.5)
        offset = torch.randn((1, 1, G, 1), generator=g, device=DEV)
        x = torch.randn((M, S, G, C // G), generator=g, device=DEV) * spread + offset
        s["x"] = x.reshape(M, S, C).to(io)
        s["weight"] = 1.0 + normal(C, dtype=torch.float32, scale=0.2)
        s["bias"] = normal(C, dtype=torch.float32, scale=0.2)
        s["z"] = normal(M, S, C) if c["gate"] else None
        if c["op"] == "norm_bwd":
            s["dy"] = normal(M, S, C)
            s["mean"], s["rstd"] = _statistics(s["x"].float(), G)
        return s
    B, H, G, K, V = c["B"], c["H"], c["G"], c["K"], c["V"]
    # decay rates spread over memories of two tokens to two thousand
    rate = torch.exp(torch.linspace(math.log(0.5), math.log(1 / 2048), H, device=DEV))
    s["log_decay"] = -rate * (0.8 + 0.4 * torch.rand(H, generator=g, device=DEV))
    s["scale"] = K ** -0.5
    if c["op"] == "step":
        s["state"] = normal(B, H, K, V, dtype=torch.float32)
        s["q"], s["k"], s["v"] = normal(B, G, K), normal(B, G, K), normal(B, H, V)
        if c["norm"]:
            s["weight"] = 1.0 + normal(H * V, dtype=torch.float32, scale=0.2)
            s["z"] = normal(B, H, V)
        return s
    L = c["L"]
    s["q"], s["k"], s["v"] = normal(B, L, G, K), normal(B, L, G, K), normal(B, L, H, V)
    s["h0"] = normal(B, H, K, V, dtype=torch.float32) if c["h0"] else None
    s["seqlens"] = None
    if c["ragged"]:
        n = torch.randint(max(1, L // 4), L + 1, (B,), generator=g, device=DEV)
        n[0] = L
        s["seqlens"] = n.to(torch.int32)
    if c["op"] == "bwd":
        s["do"] = normal(B, L, H, V)
        s["dh_final"] = normal(B, H, K, V, dtype=torch.float32, scale=0.1) if c["h0"] else None
    return s


# ------------------------------------------------------------------ the plain forms
def _statistics(x, G):
    """mean and 1 / sqrt(variance + EPS) per sample and group of x [M, S, C] (32 bits)."""
    M, S, C = x.shape
    xg = x.reshape(M, S, G, C // G)
    mean = xg.mean(dim=(1, 3))
    var = (xg - mean[:, None, :, None]).square().mean(dim=(1, 3))
    return mean, torch.rsqrt(var + EPS)


def _plain_norm(s):
    c = s["case"]
    M, S, C, G = c["M"], c["S"], c["C"], c["groups"]
    x = s["x"].float()
    mean, rstd = _statistics(x, G)
    xhat = ((x.reshape(M, S, G, C // G) - mean[:, None, :, None]) * rstd[:, None, :, None]).reshape(M, S, C)
    u = xhat * s["weight"] + s["bias"]
    y = u * torch.sigmoid(u) if c["act"] == "silu" else u
    if s["z"] is not None:
        z = s["z"].float()
        y = y * z * torch.sigmoid(z)
    return y.to(s["x"].dtype), mean, rstd


def _plain_norm_bwd(s):
    c = s["case"]
    M, S, C, G = c["M"], c["S"], c["C"], c["groups"]
    io = s["x"].dtype
    rstd = s["rstd"][:, None, :, None]
    xhat = ((s["x"].float().reshape(M, S, G, C // G) - s["mean"][:, None, :, None]) * rstd).reshape(M, S, C)
    u = xhat * s["weight"] + s["bias"]
    du = s["dy"].float()
    dz = None
    if s["z"] is not None:
        z = s["z"].float()
        sz = torch.sigmoid(z)
        su = torch.sigmoid(u) if c["act"] == "silu" else 1.0
        dz = (du * (u * su) * (sz * (1 + z * (1 - sz)))).to(io)
        du = du * (z * sz)
    if c["act"] == "silu":
        su = torch.sigmoid(u)
        du = du * (su * (1 + u * (1 - su)))
    dw, db = (du * xhat).sum(dim=(0, 1)), du.sum(dim=(0, 1))
    dn = (du * s["weight"]).reshape(M, S, G, C // G)
    xg = xhat.reshape(M, S, G, C // G)
    dx = rstd * (dn - dn.mean(dim=(1, 3), keepdim=True) - xg * (dn * xg).mean(dim=(1, 3), keepdim=True))
    return {"dx": dx.reshape(M, S, C).to(io), "dweight": dw, "dbias": db, "dz": dz}


def _heads(t, H):
    """[B, L, G, K] -> [B, H, L, K] in 32 bits, each group repeated for its heads."""
    B, L, G, K = t.shape
    return t.float()[:, :, :, None, :].expand(B, L, G, H // G, K).reshape(B, L, H, K).transpose(1, 2).contiguous()


def _powers(a, n):
    """lam^n for every head, [H, *n.shape], n >= 0."""
    return torch.exp(a.double().reshape(-1, *([1] * n.dim())) * n).float()


def _mix(q, k, v, a):
    """sum_{j <= i} lam^(i-j) (q_i . k_j) v_j for [B, H, L, .] in 32 bits, by chunks."""
    B, H, L, _ = q.shape
    C = CHUNK
    n = -(-L // C)
    pad = n * C - L
    q, k, v = (torch.nn.functional.pad(t, (0, 0, 0, pad)).reshape(B, H, n, C, t.shape[-1]) for t in (q, k, v))
    i = torch.arange(C, device=q.device)
    lag = i[:, None] - i[None, :]
    D = _powers(a, lag.clamp(min=0).double()) * (lag >= 0)
    out = torch.matmul(torch.matmul(q, k.transpose(-1, -2)) * D[None, :, None], v)
    wk = k * _powers(a, (C - 1 - i).double())[None, :, None, :, None]
    A = torch.matmul(wk.transpose(-1, -2), v)  # what each chunk adds to the state
    m = torch.arange(n, device=q.device)
    gap = m[:, None] - 1 - m[None, :]
    W = _powers(a, (C * gap.clamp(min=0)).double()) * (gap >= 0)
    S = torch.matmul(W[None], A.reshape(B, H, n, -1)).reshape(A.shape)  # the state entering each chunk
    out = out + torch.matmul(q * _powers(a, (i + 1).double())[None, :, None, :, None], S)
    return out.reshape(B, H, n * C, -1)[:, :, :L]


def _lengths(s, B, L, device):
    """lengths [B], the rows that count [B, 1, L, 1], and the steps left after each row [B, 1, L]."""
    n = torch.full((B,), L, device=device) if s["seqlens"] is None else s["seqlens"].long()
    t = torch.arange(L, device=device)
    left = n[:, None] - 1 - t[None, :]
    return n, (left >= 0)[:, None, :, None], left.clamp(min=0)[:, None, :]


def _plain_fwd(s):
    c = s["case"]
    B, L, H = c["B"], c["L"], c["H"]
    a, scale, h0 = s["log_decay"], s["scale"], s["h0"]
    n, rows, left = _lengths(s, B, L, a.device)
    q, k = _heads(s["q"], H) * rows, _heads(s["k"], H) * rows
    v = _heads(s["v"], H) * rows
    o = _mix(q, k, v, a)
    tail = torch.exp(a.double()[None, :, None] * left).float()[..., None]  # lam^(len-1-j), [B, H, L, 1]
    h = torch.matmul((k * tail).transpose(-1, -2), v)
    if h0 is not None:
        t1 = torch.arange(1, L + 1, device=a.device).double()
        o = o + torch.matmul(q * _powers(a, t1)[None, :, :, None], h0)
        h = h + torch.exp(a.double()[None, :] * n[:, None]).float()[:, :, None, None] * h0
    return (o * scale).transpose(1, 2).to(s["v"].dtype).contiguous(), h


def _plain_bwd(s):
    c = s["case"]
    B, L, H, G = c["B"], c["L"], c["H"], c["G"]
    a, scale, h0, T = s["log_decay"], s["scale"], s["h0"], s["dh_final"]
    io = s["v"].dtype
    n, rows, left = _lengths(s, B, L, a.device)
    q, k = _heads(s["q"], H) * rows * scale, _heads(s["k"], H) * rows
    v, do = _heads(s["v"], H) * rows, _heads(s["do"], H) * rows
    t1 = _powers(a, torch.arange(1, L + 1, device=a.device).double())[None, :, :, None]  # lam^(i+1)
    dq = _mix(do, v, k, a)
    dk = _mix(v.flip(2), do.flip(2), q.flip(2), a).flip(2)
    dv = _mix(k.flip(2), q.flip(2), do.flip(2), a).flip(2)
    dh0 = torch.matmul((q * t1).transpose(-1, -2), do)
    if h0 is not None:
        dq = dq + torch.matmul(do * t1, h0.transpose(-1, -2))
    if T is not None:
        tail = torch.exp(a.double()[None, :, None] * left).float()[..., None] * rows
        dk = dk + torch.matmul(v * tail, T.transpose(-1, -2))
        dv = dv + torch.matmul(k * tail, T)
        dh0 = dh0 + torch.exp(a.double()[None, :] * n[:, None]).float()[:, :, None, None] * T

    def shared(t):  # [B, H, L, K] -> [B, L, G, K]
        return t.reshape(B, G, H // G, L, -1).sum(2).transpose(1, 2).to(io).contiguous()

    return {"dq": shared(dq * scale), "dk": shared(dk), "dv": dv.transpose(1, 2).to(io).contiguous(), "dh0": dh0}


def _plain_step(s):
    c = s["case"]
    B, H, G, K, V = c["B"], c["H"], c["G"], c["K"], c["V"]
    io = s["v"].dtype
    q, k = (s[n].float()[:, :, None, :].expand(B, G, H // G, K).reshape(B, H, K) for n in ("q", "k"))
    v = s["v"].float()
    S = s["state"]
    S.mul_(torch.exp(s["log_decay"])[None, :, None, None]).add_(k[..., :, None] * v[..., None, :])
    o = torch.matmul(q[..., None, :], S)[..., 0, :] * s["scale"]
    if c["norm"]:
        mean = o.mean(-1, keepdim=True)
        rstd = torch.rsqrt((o - mean).square().mean(-1, keepdim=True) + EPS)
        z = s["z"].float()
        o = (o - mean) * rstd * s["weight"].reshape(H, V) * z * torch.sigmoid(z)
    return o.to(io), S


# ------------------------------------------------------------------ one pass
def run(s):
    c = s["case"]
    if not own:
        return {"fwd": _plain_fwd, "bwd": _plain_bwd, "step": _plain_step, "norm": _plain_norm,
                "norm_bwd": _plain_norm_bwd}[c["op"]](s)
    import selective_scan_amd as ssa
    if c["op"] == "fwd":
        return ssa.ssm_linattn_fwd(s["q"], s["k"], s["v"], s["log_decay"], scale=s["scale"], seqlens=s["seqlens"],
                                   h0=s["h0"])
    if c["op"] == "bwd":
        return ssa.ssm_linattn_bwd(s["q"], s["k"], s["v"], s["log_decay"], s["do"], scale=s["scale"],
                                   seqlens=s["seqlens"], h0=s["h0"], dh_final=s["dh_final"])
    if c["op"] == "step":
        if not c["norm"]:
            return ssa.ssm_linattn_step(s["state"], s["q"], s["k"], s["v"], s["log_decay"],
                                        scale=s["scale"]), s["state"]
        return ssa.ssm_linattn_step(s["state"], s["q"], s["k"], s["v"], s["log_decay"], scale=s["scale"],
                                    norm_eps=EPS, norm_weight=s["weight"], z=s["z"]), s["state"]
    if c["op"] == "norm":
        return ssa.ssm_group_norm_fwd(s["x"], c["groups"], s["weight"], s["bias"], s["z"], eps=EPS, act=c["act"])
    return ssa.ssm_group_norm_bwd(s["x"], c["groups"], s["mean"], s["rstd"], s["dy"], s["weight"], s["bias"], s["z"],
                                  act=c["act"])


def work(case):
    c = case
    es = 2 if c["io"] == "bf16" else 4
    if c["op"] in ("norm", "norm_bwd"):
        n = c["M"] * c["S"] * c["C"]
        if c["op"] == "norm":
            return {"bytes": n * es * (3 if c["gate"] else 2) + 8 * c["C"] + 8 * c["M"] * c["groups"], "flops": 10 * n}
        return {"bytes": n * es * (5 if c["gate"] else 3) + 16 * c["C"] + 8 * c["M"] * c["groups"], "flops": 20 * n}
    B, H, G, K, V = c["B"], c["H"], c["G"], c["K"], c["V"]
    state = 4 * B * H * K * V
    if c["op"] == "step":
        return {"bytes": 2 * state + B * es * (2 * G * K + (3 if c["norm"] else 2) * H * V) + 4 * H,
                "flops": 4 * B * H * K * V}
    rows = B * c["L"]
    if c["op"] == "fwd":
        return {"bytes": rows * es * (2 * G * K + 2 * H * V) + state * (2 if c["h0"] else 1) + 4 * H,
                "flops": 4 * rows * H * K * V}
    return {"bytes": rows * es * (4 * G * K + 3 * H * V) + state * (3 if c["h0"] else 1) + 4 * H,
            "flops": 12 * rows * H * K * V}


# ------------------------------------------------------------------ 64 bits
def _exact_norm(s):
    c = s["case"]
    M, S, C, G = c["M"], c["S"], c["C"], c["groups"]
    x = s["x"].double().view(M, S, G, C // G).permute(0, 2, 1, 3)
    w, b = (s[n].double().view(1, G, 1, C // G) for n in ("weight", "bias"))

    def back(t):
        return t.permute(0, 2, 1, 3).reshape(M, S, C)

    gate = None if s["z"] is None else s["z"].double().view(M, S, G, C // G).permute(0, 2, 1, 3)
    if c["op"] == "norm":
        var, mean = torch.var_mean(x, dim=(2, 3), correction=0, keepdim=True)
        u = (x - mean) / torch.sqrt(var + EPS) * w + b
        y = u / (1 + torch.exp(-u)) if c["act"] == "silu" else u
        if gate is not None:
            y = y * gate / (1 + torch.exp(-gate))
        return back(y), mean[:, :, 0, 0], 1 / torch.sqrt(var + EPS)[:, :, 0, 0]
    rstd = s["rstd"].double()[:, :, None, None]
    xhat = (x - s["mean"].double()[:, :, None, None]) * rstd
    u = xhat * w + b
    d = s["dy"].double().view(M, S, G, C // G).permute(0, 2, 1, 3)
    value, slope = u, 1.0
    if c["act"] == "silu":
        e = 1 / (1 + torch.exp(-u))
        value, slope = u * e, e + u * e * (1 - e)
    dz = None
    if gate is not None:
        e = 1 / (1 + torch.exp(-gate))
        dz = back(d * value * (e + gate * e * (1 - e)))
        d = d * gate * e
    d = d * slope
    dw, db = (d * xhat).sum(dim=(0, 2)).reshape(C), d.sum(dim=(0, 2)).reshape(C)
    d = d * w
    N = S * (C // G)
    dx = rstd * (d - d.sum(dim=(2, 3), keepdim=True) / N - xhat * (d * xhat).sum(dim=(2, 3), keepdim=True) / N)
    return {"dx": back(dx), "dweight": dw, "dbias": db, "dz": dz}


def _exact_linattn(s):
    """Every pair of steps, one (sequence, head) at a time."""
    c = s["case"]
    B, L, H, G, K, V = c["B"], c["L"], c["H"], c["G"], c["K"], c["V"]
    bwd = c["op"] == "bwd"
    f64 = dict(dtype=torch.float64, device=DEV)
    o = torch.zeros((B, L, H, V), **f64)
    state = torch.zeros((B, H, K, V), **f64)
    dq, dk = (torch.zeros((B, L, G, K), **f64) for _ in range(2))
    for h in range(H):
        g = h // (H // G)
        a = s["log_decay"][h].double()
        t = torch.arange(L, **f64)
        lag = t[:, None] - t[None, :]
        D = torch.where(lag >= 0, torch.exp(a * lag.clamp(min=0)), torch.zeros((), **f64))
        for b in range(B):
            n = L if s["seqlens"] is None else int(s["seqlens"][b])
            q, k, v = s["q"][b, :n, g].double() * s["scale"], s["k"][b, :n, g].double(), s["v"][b, :n, h].double()
            into, out = torch.exp(a * (t[:n] + 1))[:, None], torch.exp(a * (n - 1 - t[:n]))[:, None]
            start = None if s["h0"] is None else s["h0"][b, h].double()
            Dn = D[:n, :n]
            P = (q @ k.t()) * Dn
            if not bwd:
                y = P @ v
                end = k.t() @ (out * v)
                if start is not None:
                    y = y + into * (q @ start)
                    end = end + torch.exp(a * n) * start
                o[b, :n, h], state[b, h] = y, end
                continue
            do = s["do"][b, :n, h].double()
            dP = (do @ v.t()) * Dn
            gq, gk, gv = dP @ k, dP.t() @ q, P.t() @ do
            g0 = q.t() @ (into * do)
            if start is not None:
                gq = gq + into * (do @ start.t())
            if s["dh_final"] is not None:
                T = s["dh_final"][b, h].double()
                gk, gv, g0 = gk + out * (v @ T.t()), gv + out * (k @ T), g0 + torch.exp(a * n) * T
            dq[b, :n, g] += gq * s["scale"]
            dk[b, :n, g] += gk
            o[b, :n, h], state[b, h] = gv, g0
    return {"dq": dq, "dk": dk, "dv": o, "dh0": state} if bwd else (o, state)


def _exact_step(s):
    c = s["case"]
    r = c["H"] // c["G"]
    q, k = (s[n].double().repeat_interleave(r, dim=1) for n in ("q", "k"))
    S = s["state"].double() * torch.exp(s["log_decay"].double()).view(1, -1, 1, 1)
    S = S + k.unsqueeze(3) * s["v"].double().unsqueeze(2)
    o = (q.unsqueeze(3) * S).sum(2) * s["scale"]
    if c["norm"]:
        var, mean = torch.var_mean(o, dim=2, correction=0, keepdim=True)
        z = s["z"].double()
        o = (o - mean) / torch.sqrt(var + EPS) * s["weight"].double().view(1, c["H"], c["V"]) * z / (1 + torch.exp(-z))
    return o, S


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("norm", "norm_bwd"):
        return _exact_norm(s)
    return _exact_step(s) if case["op"] == "step" else _exact_linattn(s)
