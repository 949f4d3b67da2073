"""Residual add with layer norm or RMS norm and dropout, its gradient, and dropout alone on the
GPU against their 64-bit definitions; and a residual block of them with the gated linear
recurrence, whose gradient is autograd's."""
import pytest
import torch

import glr_ref as ref
import selective_scan_amd as ssa
from gpu_util import DEV

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
RNG = (0x123456789ABCDEF, 2 ** 33 + 5)


def rng_tensor(v=RNG):
    return torch.tensor(v, dtype=torch.int64, device=DEV)


def make(M, C, dtype, res, seed, offset=1.0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    return dict(x=r(M, C).to(dtype), residual=None if res is None else (2 * r(M, C) + offset * r(1, C)).to(res),
                w=1 + 0.3 * r(C), b=r(C), dy=r(M, C).to(dtype), dsum=None if res is None else r(M, C).to(res))


def check(t, norm, p, what=""):
    M, C = t["x"].shape
    dt, rt = t["x"].dtype, t["x"].dtype if t["residual"] is None else t["residual"].dtype
    f = ref.factor(p, RNG, M, C)
    d = {k: None if v is None else v.to(DEV) for k, v in t.items()}
    rng = rng_tensor() if p else None
    y, s, mean, rstd = ssa.ssm_add_norm_fwd(d["x"], d["residual"], d["w"], d["b"], norm=norm, p=p, rng=rng)
    torch.cuda.synchronize()
    ry, rs, rm, rr = ref.add_norm_fwd(t["x"], t["residual"], t["w"], t["b"], 1e-5, norm, f)
    # s: the kept element's scaling and the sum, two roundings
    mag = (t["x"].double() * f).abs() + (0 if t["residual"] is None else t["residual"].double().abs())
    es = 2.0 ** -23 * mag
    ref.close(s, rs, es, 1.0, what + " sum", store=rt)
    e = ref.sum_error(C) + 2.0 ** -22
    mabs = mag.mean(-1, keepdim=True)
    w, b = t["w"].double().abs(), 0 if t["b"] is None else t["b"].double().abs()
    if norm == "layer":
        ref.close(mean, rm[:, 0], e * mabs[:, 0], 1.0, what + " mean", store=F32)
        off = (e * mabs + es) * rr                                      # of (s - mean), in units of the deviation
    else:
        assert mean is None
        off = es * rr
    # squares of values that are off: relative 2 (off rms) + the sum's
    rel = (off ** 2).mean(-1, keepdim=True).sqrt() + e
    ref.close(rstd, rr[:, 0], rr[:, 0] * rel[:, 0], 1.0, what + " rstd", store=F32)
    xhat = (rs - rm) * rr
    ex = off + xhat.abs() * (rel + 2.0 ** -22)
    ref.close(y, ry, w * ex + 2.0 ** -23 * (w * xhat.abs() + b), 1.0, what + " y", store=dt)

    # the gradient takes the sum and the statistics it is given
    m32, r32 = (None if norm == "rms" else rm[:, 0].float()), rr[:, 0].float()
    sg = rs.to(rt)
    md = None if m32 is None else m32.to(DEV)
    g = ssa.ssm_add_norm_bwd(sg.to(DEV), md, r32.to(DEV), d["dy"], d["w"], d["dsum"], norm=norm, p=p, rng=rng)
    torch.cuda.synchronize()
    r = ref.add_norm_bwd(sg, m32, r32, t["dy"], t["w"], t["dsum"], norm, f)
    m64, r64 = (0 if m32 is None else m32.double()[:, None]), r32.double()[:, None]
    xh = (sg.double() - m64) * r64
    oh = 2.0 ** -22 * (sg.double().abs() + abs(m64)) * r64              # of xhat
    dn = (t["dy"].double() * t["w"].double()).abs()
    ec = ref.sum_error(C) + 2.0 ** -22
    mean_ = lambda v: v.mean(-1, keepdim=True)  # noqa: E731
    inner = mean_(dn * xh.abs())
    eds = r64 * (2.0 ** -21 * (dn + mean_(dn) + xh.abs() * inner) + ec * mean_(dn) + oh * inner
                 + xh.abs() * mean_(dn * (oh + ec * xh.abs()))) + 2.0 ** -23 * r["dresidual"].abs()
    if t["dsum"] is not None:
        eds = eds + 2.0 ** -23 * t["dsum"].double().abs()
    ref.close(g["dresidual"], r["dresidual"], eds, 1.0, what + " dresidual", store=rt)
    ref.close(g["dx"], r["dx"], (eds + 2.0 ** -23 * r["dresidual"].abs()) * f, 1.0, what + " dx", store=dt)
    em = ref.sum_error(M)
    dy = t["dy"].double().abs()
    ref.close(g["dbias"], r["dbias"], (em * dy).sum(0), 1.0, what + " dbias", store=F32)
    ref.close(g["dweight"], r["dweight"], (dy * (oh + (em + 2.0 ** -22) * xh.abs())).sum(0), 1.0, what + " dweight",
              store=F32)


SHAPES = [(1, 1), (5, 2), (3, 7), (2, 8), (9, 63), (4, 128), (33, 129), (7, 200), (3, 511), (6, 512), (5, 520), (2, 1001),
          (130, 256), (17, 1536), (3, 2048), (4, 2049), (3, 4096), (2, 5000), (3, 8192), (2, 9001), (2, 16384)]


@pytest.mark.parametrize("types", [(BF16, BF16), (BF16, F32), (F32, F32), (BF16, None)], ids=str)
@pytest.mark.parametrize("norm,p", [("layer", 0.0), ("rms", 0.3), ("layer", 0.1)])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_forward_and_gradient(shape, norm, p, types):
    check(make(*shape, *types, seed=sum(shape)), norm, p, what=f"{shape} {norm} {p} {types}")


def test_many_rows():
    check(make(5000, 40, BF16, F32, seed=1), "layer", 0.0)
    check(make(3001, 129, F32, F32, seed=2), "rms", 0.0)


@pytest.mark.parametrize("norm", ["layer", "rms"])
def test_a_large_common_offset(norm):
    """Values 300 times their spread: a difference of large sums would lose the variance."""
    t = make(4, 1000, F32, F32, seed=5)
    t["residual"] = t["residual"] + 300.0
    check(t, norm, 0.0)


def test_rows_of_zeros_and_rows_that_are_not_finite():
    t = make(6, 96, BF16, F32, seed=6)
    t["x"][1], t["residual"][1] = 0, 0
    t["x"][3, 5] = float("nan")
    t["residual"][4, 7] = float("inf")
    d = {k: v.to(DEV) for k, v in t.items()}
    for norm in ("layer", "rms"):
        y, s, mean, rstd = ssa.ssm_add_norm_fwd(d["x"], d["residual"], d["w"], d["b"], norm=norm)
        torch.cuda.synchronize()
        assert torch.equal(y[1], d["b"].to(BF16)) and torch.isnan(y[3]).all()
        assert torch.isfinite(y[[0, 1, 2, 5]]).all()
        g = ssa.ssm_add_norm_bwd(s, mean, rstd, d["dy"], d["w"], d["dsum"], norm=norm)
        torch.cuda.synchronize()
        assert torch.isfinite(g["dx"][[0, 1, 2, 5]]).all() and torch.isnan(g["dx"][3]).all()


def test_a_dropped_element_that_is_not_finite_is_zero():
    x = torch.full((4, 64), float("nan"), device=DEV)
    y = ssa.ssm_dropout(x, 0.5, rng_tensor())
    keep = ref.bits(*RNG, 4, 64).to(DEV) >= 32768
    assert torch.isnan(y[keep]).all() and (y[~keep] == 0).all()


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("shape", [(1, 1), (3, 7), (5, 8), (17, 100), (2, 1001), (64, 512), (1, 20000)], ids=str)
def test_dropout(shape, dtype):
    M, C = shape
    x = torch.randn(shape, generator=torch.Generator().manual_seed(3)).to(dtype)
    for p in (0.0, 1e-6, 0.1, 0.5, 0.99998):
        for rng in (RNG, (-3, -1), (0, 2 ** 63 - 1)):
            y = ssa.ssm_dropout(x.to(DEV), p, rng_tensor(rng))
            torch.cuda.synchronize()
            ref.close(y, x.double() * ref.factor(p, rng, M, C), x.double().abs() * 2.0 ** -24, 1.0, str((p, rng)), store=dtype)


def test_dropout_keeps_its_share_and_offsets_continue():
    """Of n draws the share that is kept is within five deviations of 1 - p; rows drawn by two
    calls, the second from the first's end, are those of one call."""
    M, C, p = 400, 1000, 0.1
    x = torch.ones((M, C), device=DEV)
    y = ssa.ssm_dropout(x, p, rng_tensor((11, 0)))
    kept = float((y != 0).float().mean())
    assert abs(kept - 0.9) < 5 * (0.09 / (M * C)) ** 0.5 + 2.0 ** -16
    head = ssa.ssm_dropout(x[:150], p, rng_tensor((11, 0)))
    tail = ssa.ssm_dropout(x[150:], p, rng_tensor((11, ssa.ssm_dropout_blocks(150, C))))
    assert torch.equal(torch.cat([head, tail]), y)
    other = ssa.ssm_dropout(x, p, rng_tensor((12, 0)))
    both = float(((y == 0) & (other == 0)).float().mean())
    assert abs(both - 0.01) < 5 * (0.01 / (M * C)) ** 0.5 + 2.0 ** -16
    # the same mask in the fused form
    z = torch.zeros((M, C), device=DEV)
    s = ssa.ssm_add_norm_fwd(x, z, p=p, rng=rng_tensor((11, 0)))[1]
    assert torch.equal(s, y)


@pytest.mark.parametrize("C", [96, 101, 3000])
def test_in_place(C):
    t = make(70, C, BF16, F32, seed=8)
    d = {k: v.to(DEV) for k, v in t.items()}
    y, s, mean, rstd = ssa.ssm_add_norm_fwd(d["x"], d["residual"], d["w"], d["b"], p=0.2, rng=rng_tensor())
    g = ssa.ssm_add_norm_bwd(s, mean, rstd, d["dy"], d["w"], d["dsum"], p=0.2, rng=rng_tensor())
    x, res, ds = d["x"].clone(), d["residual"].clone(), d["dsum"].clone()
    y2, s2, *_ = ssa.ssm_add_norm_fwd(x, res, d["w"], d["b"], p=0.2, rng=rng_tensor(), y=x, sum=res)
    g2 = ssa.ssm_add_norm_bwd(s, mean, rstd, d["dy"], d["w"], ds, p=0.2, rng=rng_tensor(), out=dict(dresidual=ds))
    z = d["x"].clone()
    ssa.ssm_dropout(z, 0.2, rng_tensor(), y=z)
    torch.cuda.synchronize()
    assert y2 is x and s2 is res and torch.equal(x, y) and torch.equal(res, s)
    assert torch.equal(ds, g["dresidual"]) and all(torch.equal(g[k], g2[k]) for k in g)
    assert torch.equal(z, ssa.ssm_dropout(d["x"], 0.2, rng_tensor()))


def test_shapes_and_what_is_not_wanted():
    t = make(12, 40, BF16, F32, seed=9)
    d = {k: v.to(DEV) for k, v in t.items()}
    x3 = d["x"].reshape(3, 4, 40)
    y, s, mean, rstd = ssa.ssm_add_norm_fwd(x3, weight=d["w"])
    assert s is x3 and mean.shape == rstd.shape == (3, 4) and y.shape == x3.shape
    g = ssa.ssm_add_norm_bwd(s, mean, rstd, x3, d["w"], want_dresidual=False, want_dbias=False)
    assert g["dresidual"] is None and g["dbias"] is None and g["dx"].shape == x3.shape
    only = ssa.ssm_add_norm_bwd(s, mean, rstd, x3, d["w"], want_dx=False, want_dweight=False)
    assert only["dx"] is None and only["dweight"] is None and torch.equal(only["dresidual"], g["dx"])
    assert ssa.ssm_add_norm_fwd(x3, d["residual"].reshape(3, 4, 40), want_sum=False)[1] is None
    over = x3.clone()
    y4, s4, *_ = ssa.ssm_add_norm_fwd(over, weight=d["w"], y=over)
    assert y4 is over and torch.equal(s4, x3) and torch.equal(y4, y)
    e = torch.empty((0, 40), dtype=BF16, device=DEV)
    y, s, mean, rstd = ssa.ssm_add_norm_fwd(e, weight=d["w"])
    g = ssa.ssm_add_norm_bwd(e, mean, rstd, e, d["w"])
    assert y.shape == (0, 40) and (g["dweight"] == 0).all() and (g["dbias"] == 0).all()
    assert ssa.ssm_dropout(e, 0.5, rng_tensor()).shape == (0, 40)


def test_results_repeat_bit_for_bit_on_another_stream():
    t = make(3000, 520, BF16, F32, seed=10)
    d = {k: v.to(DEV) for k, v in t.items()}
    y, s, mean, rstd = ssa.ssm_add_norm_fwd(d["x"], d["residual"], d["w"], d["b"], p=0.1, rng=rng_tensor())
    g = ssa.ssm_add_norm_bwd(s, mean, rstd, d["dy"], d["w"], d["dsum"], p=0.1, rng=rng_tensor())
    torch.cuda.synchronize()
    side, r = torch.cuda.Stream(), rng_tensor()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        y2, s2, m2, r2 = ssa.ssm_add_norm_fwd(d["x"], d["residual"], d["w"], d["b"], p=0.1, rng=r, stream=side)
        g2 = ssa.ssm_add_norm_bwd(s2, m2, r2, d["dy"], d["w"], d["dsum"], p=0.1, rng=r, stream=side)
        junk = [torch.full((1 << 20,), float("nan"), device=DEV) for _ in range(4)]
        torch.cuda.synchronize()
        assert torch.equal(y, y2) and torch.equal(s, s2) and all(torch.equal(g[k], g2[k]) for k in g)
        del junk


def test_a_captured_graph_draws_anew():
    t = make(64, 200, BF16, F32, seed=11)
    d = {k: v.to(DEV) for k, v in t.items()}
    rng = rng_tensor()
    step = ssa.ssm_dropout_blocks(64, 200)

    def work():
        y, s, mean, rstd = ssa.ssm_add_norm_fwd(d["x"], d["residual"], d["w"], d["b"], p=0.1, rng=rng)
        g = ssa.ssm_add_norm_bwd(s, mean, rstd, d["dy"], d["w"], d["dsum"], p=0.1, rng=rng)
        return [y, s, mean, rstd, *g.values(), ssa.ssm_dropout(d["x"], 0.1, rng)]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        work()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        outs = work()
        rng[1] += step
    seen = []
    for rep in range(3):
        before = rng.clone()
        want = [v.clone() for v in work()]
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert int(rng[1]) == int(before[1]) + step
        assert all(torch.equal(a, b) for a, b in zip(want, outs)), rep
        seen.append(outs[-1].clone())
        _ = seen[-1].float().sum().item()
    assert not torch.equal(seen[0], seen[1]) and not torch.equal(seen[1], seen[2])


@pytest.mark.parametrize("norm", ["layer", "rms"])
def test_a_residual_block(norm):
    """Two blocks norm -> projections -> gated recurrence -> projection -> dropout and add, as a
    training step runs them, in fp32: every gradient against autograd in 64 bits, to 2e-4 of the
    gradient's norm (each operator is off by at most some 1e-6 of its sums' sizes, and torch's
    fp32 products by 2^-24 a term over 64 terms; ten of them follow each other, and what they
    pass on is multiplied by norms of order ten)."""
    B, L, C, D, p = 2, 200, 32, 48, 0.1
    gen = torch.Generator().manual_seed(4)
    r = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
    x0, target = r(B, L, C), r(B, L, C)
    layers = [dict(w=1 + 0.1 * r(C), b=0.1 * r(C), inp=r(C, 4 * D) / C ** 0.5, A=-torch.exp(r(D) - 3),
                   out=r(D, C) / D ** 0.5) for _ in range(2)]
    final = dict(w=1 + 0.1 * r(C), b=0.1 * r(C))
    rngs = [(5, 1000 * k) for k in range(2)]

    # 64 bits, autograd
    ps = [{k: v.double().requires_grad_() for k, v in lay.items()} for lay in layers]
    pf = {k: v.double().requires_grad_() for k, v in final.items()}
    xa = x0.double().requires_grad_()

    def ln(v, w, b):
        m = v.mean(-1, keepdim=True) if norm == "layer" else 0.0
        return (v - m) / torch.sqrt(((v - m) ** 2).mean(-1, keepdim=True) + 1e-5) * w + b

    s = xa
    for q, g in zip(ps, rngs):
        x, rr, i, z = (ln(s, q["w"], q["b"]) @ q["inp"]).split(D, -1)
        k = torch.sigmoid(rr)
        a = torch.exp(q["A"] * k)
        u = torch.sqrt(1 - a * a) * torch.sigmoid(i) * x
        h, ys = torch.zeros(B, D, dtype=torch.float64), []
        for t in range(L):
            h = a[:, t] * h + u[:, t]
            ys.append(h * torch.nn.functional.silu(z[:, t]))
        f = ref.factor(p, g, B * L, C).reshape(B, L, C)
        s = s + (torch.stack(ys, 1) @ q["out"]) * f
    loss = (ln(s, pf["w"], pf["b"]) * target.double()).sum()
    leaves = [xa, *(v for q in ps for v in q.values()), *pf.values()]
    want = torch.autograd.grad(loss, leaves)

    # the framework
    dev = lambda d: {k: v.to(DEV) for k, v in d.items()}  # noqa: E731
    ls, lf, tg = [dev(lay) for lay in layers], dev(final), target.to(DEV)
    gs = [rng_tensor(g) for g in rngs]
    kw = dict(norm=norm)
    saved, res, x = [], None, x0.to(DEV)
    for n, q in enumerate(ls):
        drop = dict(p=p, rng=gs[n - 1]) if n else {}
        y, res, mean, rstd = ssa.ssm_add_norm_fwd(x, res, q["w"], q["b"], **drop, **kw)
        wide = y @ q["inp"]
        xs, rr, i, z = wide.split(D, -1)
        yr, _, states = ssa.ssm_glr_fwd(xs, rr, i, q["A"], z, want_states=True)
        x = yr @ q["out"]
        saved.append((res, mean, rstd, y, (xs, rr, i, z), states, yr))
    y, res, mean, rstd = ssa.ssm_add_norm_fwd(x, res, lf["w"], lf["b"], p=p, rng=gs[1], **kw)
    g = ssa.ssm_add_norm_bwd(res, mean, rstd, tg, lf["w"], p=p, rng=gs[1], **kw)
    got = [g["dweight"], g["dbias"]]
    dx, dres = g["dx"], g["dresidual"]
    for n in (1, 0):
        q, (res, mean, rstd, y, (xs, rr, i, z), states, yr) = ls[n], saved[n]
        dout = yr.reshape(-1, D).T @ dx.reshape(-1, C)
        gr = ssa.ssm_glr_bwd(xs, rr, states, dx @ q["out"].T, i, q["A"], z)
        dwide = torch.cat([gr["dx"], gr["dr"], gr["di"], gr["dz"]], -1)
        dinp = y.reshape(-1, C).T @ dwide.reshape(-1, 4 * D)
        drop = dict(p=p, rng=gs[n - 1]) if n else {}
        g = ssa.ssm_add_norm_bwd(res, mean, rstd, dwide @ q["inp"].T, q["w"], dres, **drop, **kw)
        dx, dres = g["dx"], g["dresidual"]
        got = [g["dweight"], g["dbias"], dinp, gr["dA"], dout] + got
    got = [dres] + got
    torch.cuda.synchronize()
    for a, b, n in zip(got, want, ["x"] + ["w", "b", "inp", "A", "out"] * 2 + ["wf", "bf"]):
        assert float((a.double().cpu() - b).norm() / b.norm()) < 2e-4, n


@pytest.mark.parametrize("C", [1, 7, 100, 129, 1001, 9001])
@pytest.mark.parametrize("types", [(BF16, F32), (F32, F32), (BF16, BF16)], ids=str)
def test_nothing_is_written_around_the_outputs(C, types):
    M = 37
    t = make(M, C, *types, seed=60)
    d = {k: v.to(DEV) for k, v in t.items()}
    r = rng_tensor()
    y, s, mean, rstd = ssa.ssm_add_norm_fwd(d["x"], d["residual"], d["w"], d["b"], p=0.2, rng=r)
    g = ssa.ssm_add_norm_bwd(s, mean, rstd, d["dy"], d["w"], d["dsum"], p=0.2, rng=r)
    want = dict(y=y, sum=s, mean=mean, rstd=rstd, **g, drop=ssa.ssm_dropout(d["x"], 0.2, r))
    bufs = {n: torch.full((v.numel() + 128,), 7.0, dtype=v.dtype, device=DEV) for n, v in want.items()}
    out = {n: b[64:64 + want[n].numel()].view(want[n].shape) for n, b in bufs.items()}
    ssa.ssm_add_norm_fwd(d["x"], d["residual"], d["w"], d["b"], p=0.2, rng=r,
                         **{n: out[n] for n in ("y", "sum", "mean", "rstd")})
    ssa.ssm_add_norm_bwd(s, mean, rstd, d["dy"], d["w"], d["dsum"], p=0.2, rng=r,
                         out={n: out[n] for n in ("dx", "dresidual", "dweight", "dbias")})
    ssa.ssm_dropout(d["x"], 0.2, r, y=out["drop"])
    torch.cuda.synchronize()
    for n, b in bufs.items():
        assert (b[:64] == 7).all() and (b[64 + want[n].numel():] == 7).all(), n
        assert torch.equal(out[n], want[n]), n
