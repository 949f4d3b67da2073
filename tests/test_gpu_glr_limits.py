"""Gated linear recurrence at the ends of its range: more workgroups than one dimension of the
grid takes (sequences of one token for 65535 batches; one channel over 2^29 steps, whose tiles
wait for one another), rows that are no whole pairs, and
decays from the fastest to none."""
import pytest
import torch

import glr_ref as ref
import selective_scan_amd as ssa
import test_gpu_glr as base
from gpu_util import DEV

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
FOLD = 1 << 22  # workgroups in the grid's first dimension


def normal(shape, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return torch.randn(shape, generator=g, device=DEV, dtype=BF16)


def test_one_token_for_as_many_batches_as_there_may_be():
    """Without a state before it a token's y is k x, dx = dy k, dr = dy x k (1 - k) and dh0 = (1 - k) dy,
    k = sigmoid(r): each a product, off by what glr_ref.py says of the gates and 2^-22. Every element."""
    B, D = 65535, 4160
    assert B * (D // 64) > FOLD
    print("inputs", flush=True)
    x, r, dy = (normal((B, 1, D), s) for s in range(3))
    print("forward", flush=True)
    y, h, states = ssa.ssm_glr_fwd(x, r, form="convex", want_states=True)
    torch.cuda.synchronize()
    print("gradient", flush=True)
    out = ssa.ssm_glr_bwd(x, r, states, dy, form="convex")
    torch.cuda.synchronize()
    assert out["di"] is out["dA"] is out["dz"] is None and int(states.count_nonzero()) == 0

    def close(got, want, e, what):
        tol = torch.finfo(got.dtype).eps / 2 * want.abs() * (1 + e) + e * want.abs() + torch.finfo(F32).tiny
        worst = float(((got.double() - want).abs() / tol).max())
        assert worst <= 1.0, (what, at, worst)

    step = 4096
    for at in range(0, B, step):
        s = slice(at, at + step)
        xs, rs, ds = (t[s, 0].double() for t in (x, r, dy))
        k, om = torch.sigmoid(rs), torch.sigmoid(-rs)
        e = ref.esig(rs) + 2.0 ** -22  # of k and of 1 - k
        close(y[s, 0], k * xs, e, "y")
        close(h[s], k * xs, e, "h_final")
        close(out["dx"][s, 0], ds * k, e, "dx")
        close(out["dr"][s, 0], ds * xs * k * om, 2 * e, "dr")
        close(out["dh0"][s], om * ds, e, "dh0")


def test_one_channel_over_more_tiles_than_one_dimension_of_the_grid_takes():
    """2^22 + 6 tiles in one chain. The gates are half open (five deviations and more of r leave a
    decay below 0.999, the mean of log a is -0.8), so that 3200 steps leave nothing of what a
    window of the sequence does not know of the steps before and behind it."""
    L, n, near = (1 << 29) + 700, 9600, 3200
    assert -(-L // 128) > FOLD
    print("inputs", flush=True)
    x, r, dy = (normal((1, L, 1), 10 + s) for s in range(3))
    print("forward", flush=True)
    y, h, states = ssa.ssm_glr_fwd(x, r, form="convex", want_states=True)
    torch.cuda.synchronize()
    print("gradient", flush=True)
    out = ssa.ssm_glr_bwd(x, r, states, dy, form="convex")
    torch.cuda.synchronize()
    assert all(torch.isfinite(v).all() for v in (y, h, states, out["dx"], out["dr"], out["dh0"]))
    # tile 2^22 starts at step 2^29; the gradient takes its tiles from the end
    for at in (0, (1 << 29) - n // 256 * 128, (L - n) // 128 * 128, 700 // 128 * 128, L // 2 // 128 * 128):
        print(at, flush=True)
        cut = lambda t: t[:, at:at + n].cpu()  # noqa: B023, E731
        m = min(n, L - at)
        t = dict(x=cut(x), r=cut(r), dy=cut(dy))
        g = ref.Glr(t, "convex", None, t["dy"])
        lo, hi = 0 if at == 0 else near, m if at + m == L else m - near
        ref.close(cut(y)[:, lo:], g.y[:, lo:], g.ey[:, lo:], 1.0, f"y at {at}", store=BF16)
        sl, got = slice(lo // 128, None), states[:, at // 128:(at + m + 127) // 128].cpu()
        ref.close(got[:, sl], g.states[:, sl], g.estates[:, sl], 1.0, f"states at {at}", store=F32)
        if at + m == L:
            ref.close(h, g.h_final, g.eh_final, 1.0, "h_final", store=F32)
        if at == 0:
            ref.close(out["dh0"], *g.out["dh0"], 1.0, "dh0", store=F32)
        for k in ("dx", "dr"):
            v, e = g.out[k]
            ref.close(cut(out[k])[:, lo:hi], v[:, lo:hi], e[:, lo:hi], 1.0, f"{k} at {at}", store=BF16)


@pytest.mark.parametrize("form", ["decay", "convex"])
def test_slices_at_odd_channels_are_the_same_to_the_bounds(form):
    """bf16 rows that are no whole pairs take other lanes, which compose a wave's steps in another
    order: other bits, to the same bounds as the contiguous call; the same slices, the same bits."""
    B, L, D = 2, 700, 66
    t = ref.glr_inputs(B, L, D, BF16, form, seed=73)
    g = ref.Glr(t, form, None, t["dy"], t["dh_final"])
    d = base.to(t)
    e = dict(d)
    for n in ("x", "r", "i", "z"):
        if d[n] is not None:
            wide = torch.zeros((B, L, D + 7), dtype=BF16, device=DEV)
            wide[..., 3:3 + D] = d[n]
            e[n] = wide[..., 3:3 + D]
    first = None
    for _ in range(2):
        y, h, states = base.fwd(e, form)
        out = base.bwd(e, states, form)
        torch.cuda.synchronize()
        ref.close(y, g.y, g.ey, 1.0, "y", store=BF16)
        ref.close(h, g.h_final, g.eh_final, 1.0, "h_final", store=F32)
        for n, (v, b) in g.out.items():
            ref.close(out[n], v, b, 1.0, n, store=F32 if n in ("dA", "dh0") else BF16)
        every = [y, h, states, *(out[n] for n in g.out)]
        assert first is None or all(torch.equal(a, b) for a, b in zip(first, every))
        first = every


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("gate", [True, False])
@pytest.mark.parametrize("seqlens", [None, [300, 137]])
def test_decays_from_the_fastest_to_none(dtype, gate, seqlens):
    """A from -2^100 to 0, the gate around where A sigmoid(r) is -1 on half of the steps, anywhere
    within 100 on the others. Beside the bounds of glr_ref.py: a below 2^-126 may be 0. Of dr that
    loses |g| (|h_{t-1}| + |x|) a |A sigmoid(r)|, where the last is at most 104 (beyond, a is below
    2^-149 and the product smaller still), and its own products as much again: 2^-126 104 (G H + 1)
    with G the largest |g| that sums of |dy silu(z)| and |dh_final| allow and H the largest |h| + |x|."""
    A = torch.tensor([-2.0 ** 100, -2.0 ** 64, -1e9, -300.0, -1.0, -1e-4, -1e-12, -1e-30, -1e-38, -1e-42, -0.0, 0.0])
    D, L = len(A), 300
    t = ref.glr_inputs(2, L, D, dtype, "decay", seed=71, gate=gate)
    gen = torch.Generator().manual_seed(72)
    around = (-A.abs().clamp(1e-20, 2.0 ** 100).log()).clamp(-80, 80) + 3 * torch.randn((2, L, D), generator=gen)
    anywhere = 200 * torch.rand((2, L, D), generator=gen) - 100
    t["r"] = torch.where(torch.rand((2, L, D), generator=gen) < 0.5, around, anywhere).to(dtype)
    t["A"] = A
    g = ref.Glr(t, "decay", seqlens, t["dy"], t["dh_final"])
    d = base.to(t)
    y, h, states = base.fwd(d, "decay", seqlens)
    out = base.bwd(d, states, "decay", seqlens)
    torch.cuda.synchronize()
    ref.close(y, g.y, g.ey, 1.0, "y", store=dtype)
    ref.close(h, g.h_final, g.eh_final, 1.0, "h_final", store=F32)
    ref.close(states, g.states, g.estates, 1.0, "states", store=F32)
    most = 1.0 if t["z"] is None else float(t["z"].abs().max())
    G = float(t["dy"].double().abs().sum(1).max()) * most + float(t["dh_final"].abs().max())
    H = float(g.magb.max()) + float(t["x"].abs().max())
    for n, (v, e) in g.out.items():
        e = e + 2.0 ** -126 * 104 * (G * H + 1) if n == "dr" else e
        ref.close(out[n], v, e, 1.0, n, store=F32 if n in ("dA", "dh0") else dtype)


def test_gates_whose_sigmoid_is_just_above_the_smallest_number():
    """sigmoid(v) down to 2^-126 (v > -87.33), where 1 - sigmoid(v) is 1: dr of a decay that brings
    sigmoid(r) back, and dz. Every value is a product (x and h0 of opposite signs: no difference in
    dr either), off by the gates' exponents, 96 2^-23 each and twice in dr: 2^-14 holds all."""
    D = 64
    v = torch.linspace(-87.33, -87.2, D)
    one = torch.ones((1, 1, D))
    d = dict(x=-one, r=v.reshape(1, 1, D), i=0 * one, z=2 * one, dy=one, h0=torch.ones((1, D)), A=torch.full((D,), -2.0 ** 100))
    d = {n: t.to(DEV) for n, t in d.items()}
    states = ssa.ssm_glr_fwd(d["x"], d["r"], d["i"], d["A"], d["z"], h0=d["h0"], want_states=True)[2]
    dr = ssa.ssm_glr_bwd(d["x"], d["r"], states, d["dy"], d["i"], d["A"], d["z"])["dr"]
    s, g = torch.sigmoid(v.double()), 2 / (1 + torch.exp(torch.tensor(-2.0, dtype=torch.float64)))
    la = -2.0 ** 100 * s
    a, m = torch.exp(la), torch.sqrt(-torch.expm1(2 * la))
    want = g * a * (1 + a * 0.5 / m) * la
    assert float((dr[0, 0].double().cpu() / want - 1).abs().max()) < 2.0 ** -14

    big = dict(d, r=0 * d["r"], z=v.reshape(1, 1, D).to(DEV), A=torch.full((D,), -1.0, device=DEV))
    y, h, states = ssa.ssm_glr_fwd(big["x"], big["r"], big["i"], big["A"], big["z"], h0=d["h0"], want_states=True)
    dz = ssa.ssm_glr_bwd(big["x"], big["r"], states, d["dy"], big["i"], big["A"], big["z"])["dz"]
    want = h[0].double().cpu() * s * (1 + v.double())
    assert float((dz[0, 0].double().cpu() / want - 1).abs().max()) < 2.0 ** -14


@pytest.mark.parametrize("form,gate", [("decay", True), ("convex", False)])
def test_whole_lines_past_the_caches(form, gate):
    """More than 256 MiB in a call, strips of whole lines: a few channels against 64 bits. Outputs that
    start off a piece of 64 bytes, inputs off a line of 128, fewer tokens: other accesses, the same bits."""
    B, L, D = 2, 16500, 1536
    t = ref.glr_inputs(B, L, D, BF16, form, seed=15, gate=gate)
    d = base.to(t)
    y, h, states = base.fwd(d, form)
    out = base.bwd(d, states, form)
    torch.cuda.synchronize()
    pick = torch.tensor([0, 1, 62, 63, 64, 700, 1471, 1472, 1534, 1535])
    few = {n: None if v is None else v[..., pick].contiguous() for n, v in t.items()}
    g = ref.Glr(few, form, None, few["dy"], few["dh_final"])
    ref.close(y[..., pick.to(DEV)], g.y, g.ey, 1.0, "y", store=BF16)
    ref.close(h[..., pick.to(DEV)], g.h_final, g.eh_final, 1.0, "h_final", store=F32)
    for n, (v, e) in g.out.items():
        ref.close(out[n][..., pick.to(DEV)], v, e, 1.0, n, store=F32 if n in ("dA", "dh0") else BF16)

    def at(v, first):
        return torch.empty(v.numel() + 64, dtype=v.dtype, device=DEV)[first:first + v.numel()].view(v.shape)

    names = [n for n in ("dx", "dr", "di", "dz") if out[n] is not None]
    y2 = base.fwd(d, form, y=at(y, 8))[0]
    out2 = base.bwd(d, states, form, out={n: at(out[n], 8) for n in names})
    e = dict(d, x=at(d["x"], 32).copy_(d["x"]))
    y3 = base.fwd(e, form)[0]
    out3 = base.bwd(e, states, form)
    torch.cuda.synchronize()
    assert torch.equal(y, y2) and torch.equal(y, y3)
    assert all(out[n] is None or (torch.equal(out[n], out2[n]) and torch.equal(out[n], out3[n])) for n in out)
    short = {n: v[:, :300].contiguous() if v is not None and v.dim() == 3 else v for n, v in d.items()}
    assert torch.equal(base.fwd(short, form)[0], y[:, :300])
