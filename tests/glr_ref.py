"""The gated linear recurrence, the residual add with norm and dropout's generator in 64 bits,
from their definitions (one step after the other), and the bounds their GPU results are held to.

Bounds of the recurrence. sigmoid(v) costs (|v| + 8) 2^-23 relative (the exponent's argument is
rounded, exp2 and 1/x are good to 2^-23), as does 1 - sigmoid(v). a = exp(A s) is then off by
|A s| (that + 2^-22) + 2^-23 relative; 1 - a^2 from its series by what t = 2 A s is off, the
series' roundings (2^-22) and its next term (4e-8), from the difference by (2 a^2 (error of a) +
2^-23) / (1 - a^2); u by half of that, the input gate's error and 2^-21. Every step adds at most
four roundings of numbers no larger than habs, the same recurrence over |u| (one in a sequential
recurrence, more where pieces of the sequence are composed): E_t = a E_{t-1} + (error of a) a
habs_{t-1} + (error of u) |u| + 2^-22 habs_t. The gradient's recurrence has the same form; its
outputs are products, whose factors' errors add up. Numbers below 2^-126 may come out as 0 (all of
their size off; a factor of two stands for that where a square root halves it). Results are rounded to storage once: half a
step, finfo.eps / 2 relative."""
import torch

from linattn_ref import close, sum_error  # noqa: F401

U = 2.0 ** -24


def sigmoid(v):
    return torch.where(v >= 0, 1 / (1 + torch.exp(-v)), torch.exp(v) / (1 + torch.exp(v)))


def esig(v):
    """0 at the infinities, where the result is exact; results below 2^-126 may be 0 (v < -86)."""
    e = torch.where(v.isinf(), 0.0, (v.abs() + 8) * 2.0 ** -23)
    return torch.where((v < -86) & ~v.isinf(), 2.0, e)


class Glr:
    """All values and bounds of one set of inputs, forward and (with dy) gradient."""

    def __init__(self, t, form, seqlens=None, dy=None, dh_final=None):
        x, r = t["x"].double(), t["r"].double()
        B, L, D = x.shape
        n = torch.full((B,), L) if seqlens is None else torch.as_tensor(seqlens).clamp(0, L)
        self.rows = rows = (torch.arange(L)[None, :] < n[:, None])[:, :, None].expand(B, L, D)
        x, r = torch.where(rows, x, 0.0), torch.where(rows, r, 0.0)
        k, om, ek, eo = sigmoid(r), sigmoid(-r), esig(r), esig(-r)
        if form == "decay":
            i = torch.where(rows, t["i"].double(), 0.0)
            A = t["A"].double()
            q, eq = sigmoid(i), esig(i)
            la = A * k
            a, m2 = torch.exp(la), -torch.expm1(2 * la)
            m = m2.sqrt()
            u = m * q * x
            ea = la.abs() * (ek + 2.0 ** -22) + 2.0 ** -23
            em2 = torch.where(2 * la > -0.13, ek + 2.0 ** -21 + 4e-8, torch.zeros_like(la))
            em2 = torch.maximum(em2, torch.where(2 * la < -0.12, (2 * a * a * ea + 2.0 ** -23) / m2, 0.0))
            em2 = torch.where(m2 > 2.0 ** -125, em2, torch.where(m2 > 0, 2.0, 0.0))
            eu = em2 / 2 + eq + 2.0 ** -21
        else:
            a, u, ea, eu = om, k * x, eo, ek + 2.0 ** -23
        a, u = torch.where(rows, a, 1.0), torch.where(rows, u, 0.0)
        ea = torch.where(rows, ea, 0.0)
        h = torch.zeros((B, D), dtype=torch.float64) if t.get("h0") is None else t["h0"].double()
        hs, mags, errs = [h], [h.abs()], [torch.zeros_like(h)]
        for s in range(L):
            live = rows[:, s]
            g, e = mags[-1], errs[-1]
            new = a[:, s] * h + u[:, s]
            mag = a[:, s] * g + u[:, s].abs()
            err = a[:, s] * e + ea[:, s] * a[:, s] * g + eu[:, s] * u[:, s].abs() + 4 * U * mag
            h = torch.where(live, new, h)
            hs.append(h)
            mags.append(torch.where(live, mag, g))
            errs.append(torch.where(live, err, e))
        self.h_final, self.eh_final = h, errs[-1]
        H, E, MG = (torch.stack(v, 1) if L else h[:, None] for v in (hs, errs, mags))
        self.before, self.eb, self.magb = H[:, :-1], E[:, :-1], MG[:, :-1]
        after, eaft = H[:, 1:], E[:, 1:]
        self.states = self.before[:, ::128]
        self.estates = self.eb[:, ::128]
        if t.get("z") is None:
            y, ey = after, eaft
        else:
            z = torch.where(rows, t["z"].double(), 0.0)
            sz, oz, ez = sigmoid(z), sigmoid(-z), esig(z)
            gz = z * sz
            y, ey = after * gz, eaft * gz.abs() + (after * gz).abs() * (ez + 2.0 ** -22)
        self.y, self.ey = torch.where(rows, y, 0.0), torch.where(rows, ey, 0.0)
        if dy is None:
            return
        dy = torch.where(rows, dy.double(), 0.0)
        e, ee = dy, torch.zeros_like(dy)
        self.out = {}
        if t.get("z") is not None:
            slope, mslope = sz * (1 + z * oz), sz * (1 + z.abs() * oz)
            self.put("dz", dy * after * slope,
                     dy.abs() * (eaft * slope.abs() + after.abs() * mslope * (2 * ez + 2.0 ** -21)))
            e, ee = dy * gz, (dy * gz).abs() * (ez + 2.0 ** -22)
        c = torch.zeros((B, D), dtype=torch.float64) if dh_final is None else dh_final.double()
        ec, mc = torch.zeros_like(c), c.abs()
        gs, egs = [None] * L, [None] * L
        for s in range(L - 1, -1, -1):
            live = rows[:, s]
            g, mg = e[:, s] + c, e[:, s].abs() + mc
            eg = ee[:, s] + ec + 4 * U * mg
            gs[s], egs[s] = torch.where(live, g, 0.0), torch.where(live, eg, 0.0)
            at = a[:, s]
            c, mc, ec = (torch.where(live, at * g, c), torch.where(live, at * mg, mc),
                         torch.where(live, at * eg + ea[:, s] * at * mg, ec))
        self.out["dh0"] = (c, ec)
        g, eg = (torch.stack(v, 1) if L else torch.zeros_like(x) for v in (gs, egs))
        b, eb = self.before, self.eb
        if form == "decay":
            dx = g * m * q
            self.put("dx", dx, eg * m * q + dx.abs() * eu)
            di = dx * x * sigmoid(-i)
            self.put("di", di, (eg * m * q + dx.abs() * (eu + esig(-i) + 2.0 ** -22)) * (x * sigmoid(-i)).abs())
            p0, p1 = a * b, torch.where(m2 > 0, a * a * q * x / m, torch.zeros_like(m))
            w = torch.where(rows, g * (p0 - p1), 0.0)
            ew = (eg * (p0.abs() + p1.abs()) + g.abs() * a * eb
                  + g.abs() * (p0.abs() + p1.abs()) * (2 * ea + em2 / 2 + eq + 2.0 ** -20))
            ew = torch.where(rows, ew, 0.0)
            self.put("dr", w * A * k * om, (ew + w.abs() * (ek + eo + 2.0 ** -21)) * (A * k * om).abs())
            dA, n = (w * k).sum(dim=(0, 1)), B * L
            mag = (g.abs() * (p0.abs() + p1.abs()) * k * rows).sum(dim=(0, 1))
            self.magA = mag  # the sum of the absolute values of dA's terms
            self.out["dA"] = (dA, ((ew + w.abs() * (ek + 2.0 ** -22)) * k).sum(dim=(0, 1)) + sum_error(n) * mag)
        else:
            self.put("dx", g * k, eg * k + (g * k).abs() * (ek + 2.0 ** -23))
            self.put("dr", g * (x - b) * k * om, (eg * (x - b).abs() + g.abs() * (
                eb + (x.abs() + b.abs()) * (ek + eo + 2.0 ** -21))) * k * om)

    def put(self, name, value, bound):
        self.out[name] = (torch.where(self.rows, value, 0.0), torch.where(self.rows, bound, 0.0))


def glr_inputs(B, L, D, dtype, form, seed, gate=True, h0=True, fast=0.7, slow=0.002):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    t = dict(x=r(B, L, D).to(dtype), r=(1.5 * r(B, L, D) - (3 if form == "convex" else 0)).to(dtype), i=None, A=None,
             z=r(B, L, D).to(dtype) if gate else None, h0=r(B, D) if h0 else None, dy=r(B, L, D).to(dtype),
             dh_final=r(B, D) if h0 else None)
    if form == "decay":
        t["i"] = (1.5 * r(B, L, D)).to(dtype)
        lo, hi = torch.tensor(slow).log(), torch.tensor(fast).log()
        t["A"] = -torch.exp(lo + (hi - lo) * torch.rand(D, generator=g))
    return t


# ------------------------------------------------------------------ dropout
def philox(seed, block):
    """The four words of one block, in Python's whole numbers."""
    m = 0xFFFFFFFF
    c, k = [block & m, (block >> 32) & m, 0, 0], [seed & m, (seed >> 32) & m]
    for _ in range(10):
        p0, p1 = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
        c = [(p1 >> 32) ^ c[1] ^ k[0], p1 & m, (p0 >> 32) ^ c[3] ^ k[1], p0 & m]
        k = [(k[0] + 0x9E3779B9) & m, (k[1] + 0xBB67AE85) & m]
    return c


def bits(seed, offset, M, C):
    """The 16 bits of every element, [M, C]."""
    n = -(-C // 8)
    out = torch.empty((M, n * 8), dtype=torch.int64)
    for r in range(M):
        row = []
        for b in range(n):
            for w in philox(seed % 2 ** 64, (offset + r * n + b) % 2 ** 64):
                row += [w & 0xFFFF, w >> 16]
        out[r] = torch.tensor(row)
    return out[:, :C]


def factor(p, rng, M, C):
    """What dropout multiplies every element by, [M, C] in 64 bits."""
    least = round(65536 * p)
    if least == 0:
        return torch.ones((M, C), dtype=torch.float64)
    return (bits(int(rng[0]), int(rng[1]), M, C) >= least).double() * (65536 / (65536 - least))


# ------------------------------------------------------------------ residual add and norm
def add_norm_fwd(x, residual, w, b, eps, norm, f):
    s = x.double() * f + (0 if residual is None else residual.double())
    mean = s.mean(-1, keepdim=True) if norm == "layer" else torch.zeros_like(s[:, :1])
    rstd = 1 / torch.sqrt(((s - mean) ** 2).mean(-1, keepdim=True) + eps)
    y = (s - mean) * rstd * (1 if w is None else w.double()) + (0 if b is None else b.double())
    return y, s, mean, rstd


def add_norm_bwd(s, mean, rstd, dy, w, dsum, norm, f):
    s, dy = s.double(), dy.double()
    xhat = (s - (0 if mean is None else mean.double()[:, None])) * rstd.double()[:, None]
    dn = dy * (1 if w is None else w.double())
    ds = dn - xhat * (dn * xhat).mean(-1, keepdim=True)
    if norm == "layer":
        ds = ds - dn.mean(-1, keepdim=True)
    ds = ds * rstd.double()[:, None] + (0 if dsum is None else dsum.double())
    return dict(dx=ds * f, dresidual=ds, dweight=(dy * xhat).sum(0), dbias=dy.sum(0))
