"""The gated linear recurrence (whole sequences, their gradient, single tokens), the residual add
with layer norm or RMS norm and dropout (forward, gradient), and dropout from a counter: cases,
inputs, the operators in plain torch operations, and their values in 64 bits.

  recurrence   h_t = a_t h_{t-1} + u_t,  y = h [silu(z)]
    decay        a = exp(A sigmoid(r)),  u = sqrt(1 - a^2) sigmoid(i) x
    convex       a = 1 - sigmoid(r),     u = sigmoid(r) x
  add and norm s = residual + dropout(x),  y = (s - mean) rstd w + b  (rms: s rstd w + b)
  dropout      keeps an element whose 16 bits of Philox-4x32-10 are at least round(65536 p)
"""
import math

import torch

own = False

DEV = "cuda"
CHUNK = 128
STATE_STEPS = 128  # the state entering every so many steps is what the training forward hands on
EPS = 1e-5
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one prompt that continues a conversation: a state is carried in, the output gated
        dict(name="glr_fwd_prompt", op="fwd", B=1, L=4096, D=1536, io="bf16", form="decay", gate=True, ragged=False, h0=True),
        # a batch of long documents
        dict(name="glr_fwd_long", op="fwd", B=8, L=32768, D=512, io="bf16", form="decay", gate=False, ragged=False, h0=False),
        # a training step's sequences
        dict(name="glr_bwd_train", op="bwd", B=4, L=4096, D=1536, io="bf16", form="decay", gate=True, ragged=False, h0=False),
        # a padded batch of odd length and width in 32 bits, with a carried state
        dict(name="glr_bwd_ragged_f32", op="bwd", B=3, L=2047, D=1001, io="f32", form="convex", gate=False, ragged=True, h0=True),
        # one user's next token
        dict(name="glr_step_one", op="step", B=1, D=1536, io="bf16", form="decay", gate=True),
        # a serving batch's next tokens
        dict(name="glr_step_batch", op="step", B=256, D=2560, io="bf16", form="decay", gate=True),
        # the norm before a layer, for a batch of single tokens
        dict(name="norm_tokens", op="norm", M=64, C=2048, io="bf16", res="f32", kind="rms", p=0.0),
        # the same over a training step's tokens, with dropout on the layer's output
        dict(name="norm_train", op="norm", M=32768, C=1536, io="bf16", res="f32", kind="layer", p=0.1),
        # its gradient
        dict(name="norm_bwd_train", op="norm_bwd", M=32768, C=1536, io="bf16", res="f32", kind="layer", p=0.1),
        # an odd width and number of tokens in 32 bits
        dict(name="norm_bwd_odd_f32", op="norm_bwd", M=4099, C=1001, io="f32", res="f32", kind="rms", p=0.0),
        # dropout of a training step's activations
        dict(name="dropout_train", op="dropout", M=32768, C=1536, io="bf16", p=0.1),
        # a small odd one in 32 bits
        dict(name="dropout_odd_f32", op="dropout", M=999, C=1001, io="f32", p=0.25),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["fwd", "fwd", "bwd", "bwd", "step", "norm", "norm_bwd", "dropout"])
    io = rng.choice(["bf16", "bf16", "f32"])
    if op in ("norm", "norm_bwd", "dropout"):
        while True:
            M, C = _log_int(rng, 1, 65536), _log_int(rng, 32, 10000)
            if rng.random() < 0.6:
                C = max(8, C // 8 * 8)
            if M * C <= 32768 * 1536 // (1 if io == "bf16" else 2):
                break
        p = rng.choice([0.0, 0.1, rng.uniform(0.01, 0.6)])
        if op == "dropout":
            return dict(op=op, M=M, C=C, io=io, p=p or 0.1)
        return dict(op=op, M=M, C=C, io=io, res=rng.choice(["bf16", "f32"]) if io == "bf16" else "f32",
                    kind=rng.choice(["layer", "rms"]), p=p)
    form, gate = rng.choice(["decay", "decay", "convex"]), rng.random() < 0.5
    D = _log_int(rng, 48, 5000)
    if rng.random() < 0.6:
        D = D // 8 * 8
    if op == "step":
        return dict(op=op, B=_log_int(rng, 1, 256), D=D, io=io, form=form, gate=gate)
    most = (8 * 32768 * 512 if op == "fwd" else 4 * 4096 * 1536) // (1 if io == "bf16" else 2)
    while True:
        B, L = _log_int(rng, 1, 16), _log_int(rng, 1, 32768)
        if B * L * D <= most:
            break
    return dict(op=op, B=B, L=L, D=D, io=io, form=form, gate=gate, ragged=rng.random() < 0.4, h0=rng.random() < 0.5)


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    c = dict(case)
    io = TYPES[c["io"]]

    def normal(*shape, dtype=io, scale=1.0, mean=0.0):
        return (torch.randn(shape, generator=g, device=DEV) * scale + mean).to(dtype)

    s = {"case": c}
    if c["op"] in ("norm", "norm_bwd", "dropout"):
        M, C = c["M"], c["C"]
        s["rng"] = torch.randint(0, 2 ** 40, (2,), generator=g, device=DEV, dtype=torch.int64)  # seed, offset
        if c["op"] == "dropout":
            s["x"] = normal(M, C)
            return s
        res = TYPES[c["res"]]
        s["weight"] = 1.0 + normal(C, dtype=torch.float32, scale=0.2)
        s["bias"] = normal(C, dtype=torch.float32, scale=0.2) if c["kind"] == "layer" else None
        # a residual stream grows wider than what a layer adds, and channels differ in their mean
        stream = torch.randn((M, C), generator=g, device=DEV) * 2 + torch.randn((1, C), generator=g, device=DEV)
        if c["op"] == "norm":
            s["x"], s["residual"] = normal(M, C), stream.to(res)
            return s
        s["sum"] = stream.to(res)
        s["dy"], s["dsum"] = normal(M, C), normal(M, C, dtype=res)
        s["mean"], s["rstd"] = _statistics(s["sum"].float(), c["kind"])
        return s
    B, D = c["B"], c["D"]
    s["A"] = s["i"] = None
    if c["form"] == "decay":
        # memories of a few tokens to a few thousand at a gate of one half
        s["A"] = -torch.exp(torch.empty(D, device=DEV).uniform_(math.log(0.002), math.log(0.7), generator=g))
    shape = (B, D) if c["op"] == "step" else (B, c["L"], D)
    s["x"] = normal(*shape)
    # a convex gate is mostly small, so that it too remembers
    s["r"] = normal(*shape, scale=1.5, mean=0.0 if c["form"] == "decay" else -3.0)
    if c["form"] == "decay":
        s["i"] = normal(*shape, scale=1.5)
    s["z"] = normal(*shape) if c["gate"] else None
    if c["op"] == "step":
        s["state"] = normal(B, D, dtype=torch.float32)
        return s
    L = c["L"]
    s["h0"] = normal(B, D, dtype=torch.float32) if c["h0"] else None
    s["seqlens"] = None
    if c["ragged"]:
        n = torch.randint(max(1, L // 4), L + 1, (B,), generator=g, device=DEV)
        n[0] = L
        s["seqlens"] = n.to(torch.int32)
    if c["op"] == "bwd":
        s["dy"] = normal(B, L, D)
        s["dh_final"] = normal(B, D, dtype=torch.float32, scale=0.5) if c["h0"] else None
        a, u = _coefficients(s)[:2]
        s["states"] = _entering(_scan(a, u, s["h0"]), s["h0"])[:, ::STATE_STEPS].contiguous()
    return s


# ------------------------------------------------------------------ the plain forms
def _silu(z):
    return z * torch.sigmoid(z)


def _silu_slope(z):
    g = torch.sigmoid(z)
    return g * (1 + z * (1 - g))


def _rows(s):
    """[B, L, 1], true in a sequence and false in its padding; None without padding."""
    if s["seqlens"] is None:
        return None
    t = torch.arange(s["case"]["L"], device=s["x"].device)
    return (t[None, :] < s["seqlens"].long()[:, None])[:, :, None]


def _coefficients(s):
    """a, u, and what the gradient needs of the gates, in 32 bits; a = 1 and u = 0 at padding."""
    x, r = s["x"].float(), s["r"].float()
    if s["case"]["form"] == "decay":
        sr, si = torch.sigmoid(r), torch.sigmoid(s["i"].float())
        l = s["A"] * sr
        m2 = -torch.expm1(2 * l)
        a, u = torch.exp(l), torch.sqrt(m2) * si * x
        more = (sr, si, m2)
    else:
        k = torch.sigmoid(r)
        a, u, more = torch.sigmoid(-r), k * x, (k,)
    rows = _rows(s) if "seqlens" in s else None
    if rows is not None:
        a, u = torch.where(rows, a, 1.0), torch.where(rows, u, 0.0)
    return a, u, more


def _scan(a, u, h0):
    """h_t = a_t h_{t-1} + u_t over dimension 1: inside every chunk, then from chunk to chunk."""
    B, L, D = a.shape
    n = -(-L // CHUNK)
    if n * CHUNK > L:
        a = torch.cat([a, a.new_ones(B, n * CHUNK - L, D)], 1)
        u = torch.cat([u, u.new_zeros(B, n * CHUNK - L, D)], 1)
    a, u = a.view(B, n, CHUNK, D), u.view(B, n, CHUNK, D)
    h = torch.empty_like(u)
    p = torch.empty_like(a)
    h[:, :, 0], p[:, :, 0] = u[:, :, 0], a[:, :, 0]
    for t in range(1, CHUNK):
        torch.addcmul(u[:, :, t], a[:, :, t], h[:, :, t - 1], out=h[:, :, t])
        torch.mul(a[:, :, t], p[:, :, t - 1], out=p[:, :, t])
    carry = torch.empty((B, n, D), dtype=torch.float32, device=a.device)
    carry[:, 0] = 0.0 if h0 is None else h0
    for k in range(1, n):
        torch.addcmul(h[:, k - 1, -1], p[:, k - 1, -1], carry[:, k - 1], out=carry[:, k])
    h.addcmul_(p, carry[:, :, None, :])
    return h.view(B, n * CHUNK, D)[:, :L]


def _entering(h, h0):
    """The state before each step."""
    first = torch.zeros_like(h[:, :1]) if h0 is None else h0[:, None]
    return torch.cat([first, h[:, :-1]], 1)


def _plain_fwd(s):
    a, u, _ = _coefficients(s)
    h = _scan(a, u, s["h0"])
    y = h if s["z"] is None else h * _silu(s["z"].float())
    rows = _rows(s)
    if rows is not None:
        y = torch.where(rows, y, 0.0)
    return y.to(s["x"].dtype), h[:, -1].contiguous()


def _plain_bwd(s):
    io = s["x"].dtype
    rows = _rows(s)
    a, u, more = _coefficients(s)
    h = _scan(a, u, s["h0"])
    before = _entering(h, s["h0"])
    e = s["dy"].float()
    dz = None
    if s["z"] is not None:
        z = s["z"].float()
        dz = e * h * _silu_slope(z)
        e = e * _silu(z)
    if rows is not None:
        e = torch.where(rows, e, 0.0)
    # g_t = e_t + a_{t+1} g_{t+1}, from the last step to the first
    T = s["dh_final"]
    later = torch.cat([a[:, 1:], torch.ones_like(a[:, :1])], 1)
    g = _scan(later.flip(1), e.flip(1), T).flip(1)
    dh0 = a[:, 0] * g[:, 0]
    x = s["x"].float()
    di = dA = None
    if s["case"]["form"] == "decay":
        sr, si, m2 = more
        m = torch.sqrt(m2)
        dx = g * m * si
        di = g * m * x * si * (1 - si)
        dl = g * (a * before - a * a * si * x / m)
        if rows is not None:
            dl = torch.where(rows, dl, 0.0)
        dA = (dl * sr).sum(dim=(0, 1))
        dr = dl * s["A"] * sr * (1 - sr)
    else:
        k = more[0]
        dx = g * k
        dr = g * (x - before) * k * torch.sigmoid(-s["r"].float())

    def out(t):
        return None if t is None else (t if rows is None else torch.where(rows, t, 0.0)).to(io)

    return {"dx": out(dx), "dr": out(dr), "di": out(di), "dA": dA, "dz": out(dz), "dh0": dh0}


def _plain_step(s):
    a, u, _ = _coefficients(s)
    h = s["state"]
    h.mul_(a).add_(u)
    y = h if s["z"] is None else h * _silu(s["z"].float())
    return y.to(s["x"].dtype), h


def _philox(rng, M, C):
    """The 16 bits of every element of [M, C]: each block of eight channels of a row takes one
    Philox-4x32-10 value (counter: offset + the block's number, key: the seed)."""
    n = -(-C // 8)
    low = 0xFFFFFFFF
    ctr = rng[1] + torch.arange(M * n, device=rng.device)
    c0, c1 = ctr & low, (ctr >> 32) & low
    c2, c3 = torch.zeros_like(c0), torch.zeros_like(c0)
    k0, k1 = rng[0] & low, (rng[0] >> 32) & low
    for _ in range(10):
        p0, p1 = c0 * 0xD2511F53, c2 * 0xCD9E8D57  # the low 64 bits, whatever their sign
        c0, c1, c2, c3 = ((p1 >> 32) & low) ^ c1 ^ k0, p1 & low, ((p0 >> 32) & low) ^ c3 ^ k1, p0 & low
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    words = torch.stack([c0, c1, c2, c3], 1)
    halves = torch.stack([words & 0xFFFF, words >> 16], 2)
    return halves.view(M, n * 8)[:, :C]


def _dropped(x, p, rng):
    """dropout(x) in 32 bits."""
    least = round(65536 * p)
    if least == 0:
        return x.float()
    keep = _philox(rng, *x.shape) >= least
    return torch.where(keep, x.float() * (65536.0 / (65536 - least)), 0.0)


def _statistics(v, kind):
    """mean (None for rms) and rstd of every row."""
    if kind == "rms":
        return None, torch.rsqrt(v.square().mean(-1) + EPS)
    mean = v.mean(-1)
    return mean, torch.rsqrt((v - mean[:, None]).square().mean(-1) + EPS)


def _plain_norm(s):
    c = s["case"]
    v = s["residual"].float() + _dropped(s["x"], c["p"], s["rng"])
    mean, rstd = _statistics(v, c["kind"])
    y = (v if mean is None else v - mean[:, None]) * rstd[:, None] * s["weight"]
    if s["bias"] is not None:
        y = y + s["bias"]
    return y.to(s["x"].dtype), v.to(s["residual"].dtype), mean, rstd


def _plain_norm_bwd(s):
    c = s["case"]
    v, dy = s["sum"].float(), s["dy"].float()
    xhat = (v if s["mean"] is None else v - s["mean"][:, None]) * s["rstd"][:, None]
    dn = dy * s["weight"]
    ds = dn - xhat * (dn * xhat).mean(-1, keepdim=True)
    if c["kind"] == "layer":
        ds = ds - dn.mean(-1, keepdim=True)
    ds = ds * s["rstd"][:, None] + s["dsum"].float()
    return {"dx": _dropped(ds, c["p"], s["rng"]).to(s["dy"].dtype), "dresidual": ds.to(s["sum"].dtype),
            "dweight": (dy * xhat).sum(0), "dbias": dy.sum(0) if c["kind"] == "layer" else None}


def _plain_dropout(s):
    return _dropped(s["x"], s["case"]["p"], s["rng"]).to(s["x"].dtype)


# ------------------------------------------------------------------ one pass
def run(s):
    c = s["case"]
    op = c["op"]
    if not own:
        return {"fwd": _plain_fwd, "bwd": _plain_bwd, "step": _plain_step, "norm": _plain_norm,
                "norm_bwd": _plain_norm_bwd, "dropout": _plain_dropout}[op](s)
    import selective_scan_amd as ssa
    if op == "fwd":
        y, h, _ = ssa.ssm_glr_fwd(s["x"], s["r"], s["i"], s["A"], s["z"], form=c["form"], seqlens=s["seqlens"],
                                  h0=s["h0"])
        return y, h
    if op == "bwd":
        return ssa.ssm_glr_bwd(s["x"], s["r"], s["states"], s["dy"], s["i"], s["A"], s["z"], form=c["form"],
                               seqlens=s["seqlens"], dh_final=s["dh_final"])
    if op == "step":
        return ssa.ssm_glr_step(s["state"], s["x"], s["r"], s["i"], s["A"], s["z"], form=c["form"]), s["state"]
    rng = s["rng"] if c["p"] else None
    if op == "norm":
        return ssa.ssm_add_norm_fwd(s["x"], s["residual"], s["weight"], s["bias"], eps=EPS, norm=c["kind"], p=c["p"],
                                    rng=rng)
    if op == "norm_bwd":
        return ssa.ssm_add_norm_bwd(s["sum"], s["mean"], s["rstd"], s["dy"], s["weight"], s["dsum"], norm=c["kind"],
                                    p=c["p"], rng=rng, want_dbias=c["kind"] == "layer")
    return ssa.ssm_dropout(s["x"], c["p"], rng)


def work(case):
    c = case
    es = 2 if c["io"] == "bf16" else 4
    if c["op"] in ("norm", "norm_bwd", "dropout"):
        n = c["M"] * c["C"]
        if c["op"] == "dropout":
            return {"bytes": 2 * n * es, "flops": 2 * n}
        rs, stats = 2 if c["res"] == "bf16" else 4, 4 * c["M"] * (2 if c["kind"] == "layer" else 1)
        vectors = 4 * c["C"] * (2 if c["kind"] == "layer" else 1)
        if c["op"] == "norm":
            return {"bytes": n * (2 * es + 2 * rs) + vectors + stats, "flops": 10 * n}
        return {"bytes": n * (2 * es + 3 * rs) + vectors + 4 * c["C"] + stats, "flops": 16 * n}
    ins, state = (3 if c["form"] == "decay" else 2) + c["gate"], 4 * c["B"] * c["D"]
    A = 4 * c["D"] if c["form"] == "decay" else 0
    if c["op"] == "step":
        n = c["B"] * c["D"]
        return {"bytes": n * es * (ins + 1) + 2 * state + A, "flops": 20 * n}
    n = c["B"] * c["L"] * c["D"]
    if c["op"] == "fwd":
        return {"bytes": n * es * (ins + 1) + state * (2 if c["h0"] else 1) + A, "flops": 20 * n}
    return {"bytes": n * es * (2 * ins + 1) + state * (3 if c["h0"] else 1) + 2 * A, "flops": 45 * n}


# ------------------------------------------------------------------ 64 bits
def _exact_gates(s):
    """Per element in 64 bits: log a, a, u and the gates."""
    x, r = s["x"].double(), s["r"].double()
    if s["case"]["form"] == "convex":
        la = -torch.nn.functional.softplus(r)
        k = 1 / (1 + torch.exp(-r))
        return la.exp(), k * x, k, None, None
    k, q = 1 / (1 + torch.exp(-r)), 1 / (1 + torch.exp(-s["i"].double()))
    la = s["A"].double() * k
    m = (-torch.expm1(2 * la)).sqrt()
    return la.exp(), m * q * x, k, q, m


def _exact_glr(s):
    """One step after the other."""
    c = s["case"]
    B, L, D = s["x"].shape
    a, u, k, q, m = _exact_gates(s)
    n = torch.full((B, 1), L, device=DEV) if s["seqlens"] is None else s["seqlens"].long()[:, None]
    h = torch.zeros((B, D), dtype=torch.float64, device=DEV) if s["h0"] is None else s["h0"].double()
    first = h
    whole = s["seqlens"] is None
    hs = torch.empty((B, L, D), dtype=torch.float64, device=DEV)
    for t in range(L):
        new = a[:, t] * h + u[:, t]
        h = new if whole else torch.where(n > t, new, h)
        hs[:, t] = h
    del u
    inside = None if whole else (torch.arange(L, device=DEV)[None] < n)[:, :, None]

    def zero(t):
        return t if inside is None else t * inside

    if c["op"] == "fwd":
        if s["z"] is not None:
            z = s["z"].double()
            hs = hs * (z / (1 + torch.exp(-z)))
        return zero(hs), h
    gate, dz = 1.0, None
    if s["z"] is not None:
        z = s["z"].double()
        e = 1 / (1 + torch.exp(-z))
        gate, dz = z * e, zero(s["dy"].double() * hs * (e + z * e * (1 - e)))
    d = s["dy"].double() * gate
    carry = torch.zeros((B, D), dtype=torch.float64, device=DEV) if s["dh_final"] is None else s["dh_final"].double()
    g = torch.zeros((B, L, D), dtype=torch.float64, device=DEV)
    for t in range(L - 1, -1, -1):
        at = d[:, t] + carry
        new = a[:, t] * at
        if whole:
            g[:, t], carry = at, new
        else:
            g[:, t], carry = torch.where(n > t, at, 0.0), torch.where(n > t, new, carry)
    prev = torch.cat([first[:, None], hs[:, :-1]], 1)
    x = s["x"].double()
    if c["form"] == "convex":
        return {"dx": g * k, "dr": g * (x - prev) * k * a, "di": None, "dA": None, "dz": dz, "dh0": carry}
    dla = g * a * (prev - a * q * x / m)
    return {"dx": g * m * q, "dr": dla * s["A"].double() * k / (1 + torch.exp(s["r"].double())),
            "di": g * m * x * q / (1 + torch.exp(s["i"].double())), "dA": (dla * k).sum(dim=(0, 1)), "dz": dz,
            "dh0": carry}


def _exact_step(s):
    a, u = _exact_gates(s)[:2]
    h = a * s["state"].double() + u
    if s["z"] is None:
        return h, h
    z = s["z"].double()
    return h * z / (1 + torch.exp(-z)), h


def _exact_keep(s):
    """What each element is multiplied by: the generator in products of 16-bit halves."""
    c = s["case"]
    M, C = s["dy" if c["op"] == "norm_bwd" else "x"].shape
    least = int(math.floor(c["p"] * 65536 + 0.5))
    if least == 0:
        return torch.ones((M, C), dtype=torch.float64, device=DEV)
    seed, offset = (int(v) for v in s["rng"].tolist())

    def product(v, const):  # (high, low) 32 bits of v * const
        lo, hi = v * (const & 0xFFFF), v * (const >> 16)
        lo, hi = (lo + ((hi & 0xFFFF) << 16)), hi >> 16
        return hi + (lo >> 32), lo & 0xFFFFFFFF

    octets = (C + 7) // 8
    number = torch.arange(M, device=DEV)[:, None] * octets + torch.arange(octets, device=DEV)[None, :] + offset
    w = [number % 2 ** 32, number // 2 ** 32, torch.zeros_like(number), torch.zeros_like(number)]
    for turn in range(10):
        key0 = (seed % 2 ** 32 + turn * 0x9E3779B9) % 2 ** 32
        key1 = (seed // 2 ** 32 + turn * 0xBB67AE85) % 2 ** 32
        h0, l0 = product(w[0], 0xD2511F53)
        h1, l1 = product(w[2], 0xCD9E8D57)
        w = [h1 ^ w[1] ^ key0, l1, h0 ^ w[3] ^ key1, l0]
    c = torch.arange(C, device=DEV)
    bits = torch.empty((M, C), dtype=torch.int64, device=DEV)
    for j in range(8):
        v = w[j // 2] // 65536 if j % 2 else w[j // 2] % 65536
        bits[:, j::8] = v[:, :bits[:, j::8].shape[1]]
    return (bits >= least).double() * (65536 / (65536 - least))


def _exact_norm(s):
    c = s["case"]
    if c["op"] == "norm":
        v = s["residual"].double() + s["x"].double() * _exact_keep(s)
        if c["kind"] == "rms":
            mean, rstd = None, (v.pow(2).sum(1) / c["C"] + EPS).pow(-0.5)
        else:
            var, mean = torch.var_mean(v, dim=1, correction=0)
            rstd = (var + EPS).pow(-0.5)
        y = (v if mean is None else v - mean[:, None]) * rstd[:, None] * s["weight"].double()
        return (y if s["bias"] is None else y + s["bias"].double()), v, mean, rstd
    v, d, r = s["sum"].double(), s["dy"].double(), s["rstd"].double()[:, None]
    hat = v * r if s["mean"] is None else (v - s["mean"].double()[:, None]) * r
    w = d * s["weight"].double()
    inner = (w * hat).sum(1, keepdim=True) / c["C"]
    ds = w - hat * inner - (w.sum(1, keepdim=True) / c["C"] if c["kind"] == "layer" else 0.0)
    ds = ds * r + s["dsum"].double()
    return {"dx": ds * _exact_keep(s), "dresidual": ds, "dweight": (d * hat).sum(0),
            "dbias": d.sum(0) if c["kind"] == "layer" else None}


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("fwd", "bwd"):
        return _exact_glr(s)
    if op == "step":
        return _exact_step(s)
    return s["x"].double() * _exact_keep(s) if op == "dropout" else _exact_norm(s)
