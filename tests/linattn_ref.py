"""Linear attention with a decay per head and the group norm in 64 bits, from their
definitions (every pair of steps; no chunks, no recurrence), and the bounds their
GPU results are held to.

Bounds. Each value r is a sum of products; m is the same sum with every factor's
absolute value, so a relative error c on every term moves r by at most c m. A term
of a linear attention output passes at most: K roundings of its score's dot product
(2^-24 each, fp32 accumulation), one per step between its place and the output in the
carried state (at most L), the chunk's own sum (at most 128) and K of the read-out;
with bf16 storage three operands formed in fp32 may enter a product as a pair of bf16
numbers, hi = round(x), lo = round(x - hi), whose sum is off by at most 2^-9 2^-9 |x|;
powers of the decay cost 2^-22. The result is rounded to storage once: half a step,
finfo.eps / 2 relative. A norm's statistics are sums of at most n terms, added in at
most n / 64 + 64 roundings; sigmoid(x) costs (|x| + 8) 2^-23 relative (the exponent's
argument is rounded, exp2 and 1/x are good to 2^-23)."""
import math

import torch


def heads(t, H):
    """[B, L, G, K] -> [B, L, H, K] in 64 bits."""
    return t.double().repeat_interleave(H // t.shape[2], dim=2)


def _lens(seqlens, B, L):
    return [L] * B if seqlens is None else [max(0, min(int(n), L)) for n in seqlens]


def _pow(a, n):
    """exp(a n) with 0 * inf = 0."""
    return torch.where(n == 0, torch.ones_like(n), torch.exp(a * n))


def fwd(q, k, v, a, scale, seqlens=None, h0=None):
    B, L, H, V = v.shape
    K = q.shape[3]
    q, k, v, a = heads(q, H), heads(k, H), v.double(), a.double()
    o = torch.zeros((B, L, H, V), dtype=torch.float64)
    hf = torch.zeros((B, H, K, V), dtype=torch.float64)
    for b, n in enumerate(_lens(seqlens, B, L)):
        t = torch.arange(n, dtype=torch.float64)
        lag = t[:, None] - t[None, :]
        for h in range(H):
            D = torch.where(lag >= 0, _pow(a[h], lag.clamp(min=0)), torch.zeros_like(lag))
            qb, kb, vb = q[b, :n, h], k[b, :n, h], v[b, :n, h]
            y = ((qb @ kb.T) * D) @ vb
            s = (kb * _pow(a[h], n - 1 - t)[:, None]).T @ vb
            if h0 is not None:
                y = y + _pow(a[h], t + 1)[:, None] * (qb @ h0[b, h].double())
                s = s + _pow(a[h], torch.tensor(float(n), dtype=torch.float64)) * h0[b, h].double()
            o[b, :n, h] = scale * y
            hf[b, h] = s
    return o, hf


def bwd(q, k, v, a, scale, dout, seqlens=None, h0=None, T=None):
    B, L, H, V = v.shape
    G, K = q.shape[2], q.shape[3]
    q, k, v, a, dout = heads(q, H), heads(k, H), v.double(), a.double(), dout.double()
    dq, dk = torch.zeros((B, L, H, K), dtype=torch.float64), torch.zeros((B, L, H, K), dtype=torch.float64)
    dv, dh0 = torch.zeros_like(v), torch.zeros((B, H, K, V), dtype=torch.float64)
    for b, n in enumerate(_lens(seqlens, B, L)):
        t = torch.arange(n, dtype=torch.float64)
        lag = t[:, None] - t[None, :]
        for h in range(H):
            D = torch.where(lag >= 0, _pow(a[h], lag.clamp(min=0)), torch.zeros_like(lag))
            qb, kb, vb, db = q[b, :n, h], k[b, :n, h], v[b, :n, h], dout[b, :n, h]
            P, dP = scale * (qb @ kb.T) * D, scale * (db @ vb.T) * D
            gq, gk, gv = dP @ kb, dP.T @ qb, P.T @ db
            into, out = _pow(a[h], t + 1)[:, None], _pow(a[h], n - 1 - t)[:, None]
            g0 = scale * (qb * into).T @ db
            if h0 is not None:
                gq = gq + scale * into * (db @ h0[b, h].double().T)
            if T is not None:
                Tb = T[b, h].double()
                gk, gv = gk + out * (vb @ Tb.T), gv + out * (kb @ Tb)
                g0 = g0 + _pow(a[h], torch.tensor(float(n), dtype=torch.float64)) * Tb
            dq[b, :n, h], dk[b, :n, h], dv[b, :n, h], dh0[b, h] = gq, gk, gv, g0
    shared = lambda g: g.reshape(B, L, G, H // G, K).sum(3)  # noqa: E731
    return dict(dq=shared(dq), dk=shared(dk), dv=dv, dh0=dh0)


def magnitude(fn, *args, **kw):
    """fn on the absolute values of its tensors (the decay's sign and lengths as they are)."""
    def f(x):
        return x.abs() if torch.is_tensor(x) and x.is_floating_point() else x
    q, k, v, a, scale, *rest = args
    return fn(f(q), f(k), f(v), a, abs(scale), *(f(x) for x in rest),
              **{n: (x if n == "seqlens" else f(x)) for n, x in kw.items()})


def term_error(L, K, V, bf16, pairs=3, extra=0):
    """Relative error of a term, from the counts above (K and V: the roles swap in the gradient)."""
    c = (2 * max(K, V) + 128 + L + extra) * 2.0 ** -24 + 2.0 ** -22
    return c + (pairs * 2.0 ** -18 if bf16 else 0.0)


def close(got, want, mag, c, what, store=None):
    """|got - want| <= c mag + half a step of the storage type ``store`` (None: that of got)."""
    dt = store or got.dtype
    g = got.detach().double().cpu()
    assert torch.isfinite(g).all(), f"{what}: not finite"
    assert g.shape == want.shape, f"{what}: shape"
    tol = torch.finfo(dt).eps / 2 * (want.abs() + c * mag) + c * mag + torch.finfo(torch.float32).tiny
    off = (g - want).abs()
    worst = float((off / tol).max()) if g.numel() else 0.0
    assert worst <= 1.0, f"{what}: {worst:.3f} times the bound"
    return worst


# ------------------------------------------------------------------ group norm
def sigmoid(x):
    return 1 / (1 + torch.exp(-x))


def norm_fwd(x, G, w=None, b=None, z=None, eps=1e-5, act="none"):
    M, S, C = x.shape
    xg = x.double().reshape(M, S, G, C // G)
    mean = xg.mean(dim=(1, 3))
    var = ((xg - mean[:, None, :, None]) ** 2).mean(dim=(1, 3))
    rstd = 1 / torch.sqrt(var + eps)
    xhat = ((xg - mean[:, None, :, None]) * rstd[:, None, :, None]).reshape(M, S, C)
    u = xhat if w is None else xhat * w.double()
    u = u if b is None else u + b.double()
    y = u * sigmoid(u) if act == "silu" else u
    y = y if z is None else y * z.double() * sigmoid(z.double())
    return y, mean, rstd


def norm_bwd(x, G, mean, rstd, dy, w=None, b=None, z=None, act="none"):
    M, S, C = x.shape
    mean, rstd = mean.double()[:, None, :, None], rstd.double()[:, None, :, None]
    xhat = ((x.double().reshape(M, S, G, C // G) - mean) * rstd).reshape(M, S, C)
    u = xhat if w is None else xhat * w.double()
    u = u if b is None else u + b.double()
    s = sigmoid(u)
    val, slope = (u * s, s * (1 + u * (1 - s))) if act == "silu" else (u, torch.ones_like(u))
    d, dz = dy.double(), None
    if z is not None:
        sz = sigmoid(z.double())
        dz = d * val * sz * (1 + z.double() * (1 - sz))
        d = d * z.double() * sz
    d = d * slope
    dw, db = (d * xhat).sum(dim=(0, 1)), d.sum(dim=(0, 1))
    dn = (d if w is None else d * w.double()).reshape(M, S, G, C // G)
    xg = xhat.reshape(M, S, G, C // G)
    dx = rstd * (dn - dn.mean(dim=(1, 3), keepdim=True) - xg * (dn * xg).mean(dim=(1, 3), keepdim=True))
    return dict(dx=dx.reshape(M, S, C), dweight=dw, dbias=db, dz=dz)


def sum_error(n):
    """Relative error (of the sum of absolute values) of a sum of n terms."""
    return (n / 64 + 64) * 2.0 ** -24


def inputs(B, L, H, G, K, V, dtype, seed, decay="mixed", h0=True, device="cpu"):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    t = dict(q=r(B, L, G, K).to(dtype), k=r(B, L, G, K).to(dtype), v=r(B, L, H, V).to(dtype),
             dout=r(B, L, H, V).to(dtype))
    if decay == "mixed":
        a = -torch.exp(torch.linspace(math.log(0.7), math.log(1e-3), H)) * (0.5 + torch.rand(H, generator=g))
    else:
        a = torch.full((H,), float(decay))
    t["log_decay"] = a
    t["h0"] = r(B, H, K, V) if h0 else None
    t["dh_final"] = r(B, H, K, V) if h0 else None
    return {n: (None if x is None else x.to(device)) for n, x in t.items()}
