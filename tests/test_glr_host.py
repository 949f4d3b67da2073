"""Gated linear recurrence, residual add with norm, and dropout without a GPU: the 64-bit forms
the GPU tests use against autograd and published values, and the refusals of the C ABI and of
the binding (all before any HIP call)."""
import ctypes

import pytest
import torch

import glr_ref as ref
import selective_scan_amd as ssa
from selective_scan_amd import ops

P = ctypes.c_void_p(0x10000)
P2 = ctypes.c_void_p(0x40000)
ODD = ctypes.c_void_p(0x10004)
ODDER = ctypes.c_void_p(0x10001)


def _recurrence(t, form, seqlens):
    """Step by step, differentiable."""
    x, r = t["x"], t["r"]
    B, L, D = x.shape
    k = torch.sigmoid(r)
    if form == "decay":
        a = torch.exp(t["A"] * k)
        u = torch.sqrt(1 - a * a) * torch.sigmoid(t["i"]) * x
    else:
        a, u = 1 - k, k * x
    h, out = t["h0"], []
    for s in range(L):
        live = torch.tensor([[s < n] for n in (seqlens or [L] * B)])
        h = torch.where(live, a[:, s] * h + u[:, s], h)
        y = h if t["z"] is None else h * torch.nn.functional.silu(t["z"][:, s])
        out.append(torch.where(live, y, 0.0))
    return torch.stack(out, 1), h


@pytest.mark.parametrize("form", ["decay", "convex"])
@pytest.mark.parametrize("gate", [True, False])
@pytest.mark.parametrize("seqlens", [None, [5, 0]])
def test_the_64_bit_recurrence_and_its_gradient_are_autograds(form, gate, seqlens):
    t = ref.glr_inputs(2, 9, 3, torch.float64, form, seed=1, gate=gate)
    t = {n: None if v is None else v.double() for n, v in t.items()}
    leaves = {n: t[n].requires_grad_() for n in ("x", "r", "i", "A", "z", "h0") if t[n] is not None}
    y, h = _recurrence(t, form, seqlens)
    want = torch.autograd.grad((y * t["dy"]).sum() + (h * t["dh_final"]).sum(), list(leaves.values()))
    with torch.no_grad():
        g = ref.Glr(t, form, seqlens, t["dy"], t["dh_final"])
        assert torch.allclose(g.y, y, atol=1e-12) and torch.allclose(g.h_final, h, atol=1e-12)
        for n, w in zip(leaves, want):
            assert torch.allclose(g.out["d" + n][0], w, atol=1e-11), n
            assert (g.out["d" + n][1] >= 0).all()


@pytest.mark.parametrize("norm", ["layer", "rms"])
@pytest.mark.parametrize("p", [0.0, 0.4])
def test_the_64_bit_norm_gradient_is_autograds(norm, p):
    gen = torch.Generator().manual_seed(2)
    r = lambda *s: torch.randn(s, generator=gen, dtype=torch.float64)  # noqa: E731
    M, C = 3, 11
    f = ref.factor(p, (7, 2 ** 40), M, C)
    x, res, w, b, dy, dsum = (v.requires_grad_() for v in (r(M, C), r(M, C), r(C), r(C), r(M, C), r(M, C)))
    y, s, mean, rstd = ref.add_norm_fwd(x, res, w, b, 1e-5, norm, f)
    s_ = x * f + res
    mu = s_.mean(-1, keepdim=True) if norm == "layer" else 0.0
    y_ = (s_ - mu) / torch.sqrt(((s_ - mu) ** 2).mean(-1, keepdim=True) + 1e-5) * w + b
    assert torch.allclose(y, y_, atol=1e-12)
    want = torch.autograd.grad((y_ * dy).sum() + (s_ * dsum).sum(), [x, res, w, b])
    got = ref.add_norm_bwd(s, mean[:, 0] if norm == "layer" else None, rstd[:, 0], dy, w, dsum, norm, f)
    for n, v in zip(("dx", "dresidual", "dweight", "dbias"), want):
        assert torch.allclose(got[n], v, atol=1e-11), n


def test_the_generator_gives_the_published_words():
    # the published known answer of Philox-4x32-10 for a zero key and counter
    assert ref.philox(0, 0) == [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]
    b = ref.bits(3, 2 ** 64 - 1, 2, 9)  # the block number goes round
    assert b.shape == (2, 9) and int(b.max()) < 65536
    assert [int(v) for v in b[0, :2]] == [ref.philox(3, 2 ** 64 - 1)[0] & 0xFFFF, ref.philox(3, 2 ** 64 - 1)[0] >> 16]
    assert int(b[0, 8]) == ref.philox(3, 0)[0] & 0xFFFF


# every case has exactly one defect, so no call reaches a launch
GDIMS = [(dict(B=0), 1), (dict(D=0), 1), (dict(io=2), 1), (dict(form=2), 1), (dict(form=-1), 1), (dict(B=65536), 2),
         (dict(D=(1 << 18) + 1, ld=(1 << 18,) * 4), 2), (dict(A=None), 1), (dict(A=ODD), 1), (dict(i=None), 1),
         (dict(form=1), 1), (dict(x=None), 1), (dict(r=None), 1), (dict(x=ODDER), 1), (dict(z=ODDER), 1),
         (dict(ld=(24, 24, 23, 0)), 1)]
GLEN = [(dict(L=-1), 1), (dict(ld=(24, (1 << 24) + 1, 24, 24)), 2), (dict(L=(1 << 30) + 1), 2), (dict(L=1 << 30, B=1, D=1 << 18), 2),
        (dict(lens=ODD), 1), (dict(ws=None, L=4096), 3), (dict(wsb=16, L=4096), 3)]


def _ld(v):
    return None if v is None else (ctypes.c_int * 4)(*v)


def _args(kw, **more):
    a = dict(B=2, L=40, D=24, io=1, form=0, x=P, r=P, i=P, A=P, z=None, ld=None, lens=None, h0=None, ws=P, wsb=1 << 40)
    a.update(more)
    a.update(kw)
    return a


def glr_fwd(**kw):
    a = _args(kw, y=ctypes.c_void_p(0x20000), hf=None, st=None)
    return ops.lib().ssm_glr_fwd(a["B"], a["L"], a["D"], a["io"], a["form"], a["x"], a["r"], a["i"], a["A"], a["z"],
                                 _ld(a["ld"]), a["lens"], a["h0"], a["y"], a["hf"], a["st"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw,status", GDIMS + [c for c in GLEN if "ws" not in c[0] and "wsb" not in c[0]] + [
    (dict(y=None), 1), (dict(y=ODD), 1), (dict(hf=ODD), 1), (dict(st=ODD), 1), (dict(h0=ODD), 1), (dict(y=P), 1),
    (dict(hf=P), 1), (dict(st=ctypes.c_void_p(0x20000)), 1)])
def test_glr_fwd_rejects(kw, status):
    assert glr_fwd(**kw) == status
    assert ops.lib().ssm_last_error().startswith(b"ssm_glr_fwd: ")


def glr_bwd(**kw):
    out = {n: ctypes.c_void_p(0x20000 + 0x1000 * k) for k, n in enumerate(("dx", "dr", "di", "dA"))}
    a = _args(kw, st=P, dy=P, dhf=None, dz=None, dh0=None, **out)
    return ops.lib().ssm_glr_bwd(a["B"], a["L"], a["D"], a["io"], a["form"], a["x"], a["r"], a["i"], a["A"], a["z"],
                                 _ld(a["ld"]), a["lens"], a["st"], a["dy"], a["dhf"], a["dx"], a["dr"], a["di"], a["dA"],
                                 a["dz"], a["dh0"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw,status", GDIMS + GLEN + [
    (dict(st=None), 1), (dict(dy=None), 1), (dict(dx=None), 1), (dict(dr=None), 1), (dict(di=None), 1),
    (dict(dA=None), 1), (dict(dz=P), 1), (dict(z=P), 1), (dict(dhf=ODD), 1), (dict(dh0=ODD), 1), (dict(dx=P), 1),
    (dict(dh0=ctypes.c_void_p(0x21000)), 1)])
def test_glr_bwd_rejects(kw, status):
    assert glr_bwd(**kw) == status
    assert ops.lib().ssm_last_error().startswith(b"ssm_glr_bwd: ")


@pytest.mark.parametrize("kw,status", GDIMS + [
    (dict(state=None), 1), (dict(y=None), 1), (dict(state=ODD), 1), (dict(y=P), 1), (dict(state=P), 1),
    (dict(B=65535, D=1 << 18), 2)])
def test_glr_step_rejects(kw, status):
    a = _args(kw, state=ctypes.c_void_p(0x20000), y=ctypes.c_void_p(0x30000))
    assert ops.lib().ssm_glr_step(a["B"], a["D"], a["io"], a["form"], a["state"], a["x"], a["r"], a["i"], a["A"], a["z"],
                                  _ld(a["ld"]), a["y"], None) == status
    assert ops.lib().ssm_last_error().startswith(b"ssm_glr_step: ")


NDIMS = [(dict(M=-1), 1), (dict(C=0), 1), (dict(io=2), 1), (dict(io=0, res=1), 1), (dict(res=3), 1), (dict(norm=2), 1),
         (dict(C=16392), 2), (dict(M=(1 << 30) + 1, C=1), 2), (dict(M=1 << 30, C=16384), 1),
         (dict(p=-0.1), 1), (dict(p=1.0), 1), (dict(p=float("nan")), 1), (dict(p=0.999999), 1),
         (dict(p=0.5, rng=None), 1), (dict(rng=ODD), 1)]


def add_norm_fwd(**kw):
    a = dict(M=4, C=24, io=1, res=0, norm=0, x=P, residual=None, w=None, b=None, eps=1e-5, p=0.0, rng=None,
             y=ctypes.c_void_p(0x20000), sum=ctypes.c_void_p(0x21000), mean=None, rstd=None)
    a.update(kw)
    return ops.lib().ssm_add_norm_fwd(a["M"], a["C"], a["io"], a["res"], a["norm"], a["x"], a["residual"], a["w"], a["b"],
                                      a["eps"], a["p"], a["rng"], a["y"], a["sum"], a["mean"], a["rstd"], None)


@pytest.mark.parametrize("kw,status", NDIMS + [
    (dict(x=None), 1), (dict(y=None), 1), (dict(eps=0.0), 1), (dict(eps=float("nan")), 1), (dict(x=ODD), 1),
    (dict(sum=ODD), 1), (dict(norm=1, mean=P), 1), (dict(sum=P), 1), (dict(mean=P), 1),
    (dict(y=P, residual=P), 1), (dict(w=ctypes.c_void_p(0x20000)), 1), (dict(sum=ctypes.c_void_p(0x20000)), 1)])
def test_add_norm_fwd_rejects(kw, status):
    assert add_norm_fwd(**kw) == status
    assert ops.lib().ssm_last_error().startswith(b"ssm_add_norm_fwd: ")


def add_norm_bwd(**kw):
    a = dict(M=4, C=24, io=1, res=0, norm=0, sum=P, w=None, mean=P, rstd=P, dy=P, dsum=None, p=0.0, rng=None,
             dx=ctypes.c_void_p(0x20000), dres=None, dw=None, db=None, ws=P, wsb=1 << 40)
    a.update(kw)
    return ops.lib().ssm_add_norm_bwd(a["M"], a["C"], a["io"], a["res"], a["norm"], a["sum"], a["w"], a["mean"], a["rstd"],
                                      a["dy"], a["dsum"], a["p"], a["rng"], a["dx"], a["dres"], a["dw"], a["db"], a["ws"],
                                      a["wsb"], None)


@pytest.mark.parametrize("kw,status", NDIMS + [
    (dict(sum=None), 1), (dict(rstd=None), 1), (dict(dy=None), 1), (dict(dx=None), 1), (dict(mean=None), 1),
    (dict(norm=1), 1), (dict(dsum=ODD), 1), (dict(dres=ODD), 1), (dict(dx=P), 1), (dict(dres=P), 1),
    (dict(dx=ctypes.c_void_p(0x30000), dsum=ctypes.c_void_p(0x30000)), 1), (dict(dw=ctypes.c_void_p(0x20000)), 1),
    (dict(ws=None, M=1000, dw=P2), 3), (dict(wsb=8, M=1000, db=P2), 3)])
def test_add_norm_bwd_rejects(kw, status):
    assert add_norm_bwd(**kw) == status
    assert ops.lib().ssm_last_error().startswith(b"ssm_add_norm_bwd: ")


@pytest.mark.parametrize("kw,status", [c for c in NDIMS if not {"res", "norm"} & set(c[0]) and c[0].get("C") != 16392] + [
    (dict(x=None), 1), (dict(y=None), 1), (dict(y=ODD), 1), (dict(C=(1 << 24) + 8), 2),
    (dict(p=0.5, rng=ctypes.c_void_p(0x20000)), 1)])
def test_dropout_rejects(kw, status):
    a = dict(M=4, C=24, io=1, x=P, p=0.0, rng=None, y=ctypes.c_void_p(0x20000))
    a.update(kw)
    assert ops.lib().ssm_dropout(a["M"], a["C"], a["io"], a["x"], a["p"], a["rng"], a["y"], None) == status
    assert ops.lib().ssm_last_error().startswith(b"ssm_dropout: ")


def test_sizes():
    assert ssa.ssm_dropout_blocks(3, 17) == 9 and ssa.ssm_dropout_blocks(1 << 30, 8) == 1 << 30
    assert ssa.ssm_glr_workspace_size(0, 4, 4) == 0 and ssa.ssm_glr_bwd_workspace_size(1, -1, 4) == 0
    assert ssa.ssm_glr_bwd_workspace_size(2, 4096, 512) > 0
    assert ssa.ssm_add_norm_bwd_workspace_size(8, 20000) == 0 and ssa.ssm_add_norm_bwd_workspace_size(8, 2000) > 0


def test_the_binding_checks_its_tensors():
    t = ref.glr_inputs(1, 6, 8, torch.float32, "decay", seed=0)
    x, r, i, A, z = (t[n] for n in ("x", "r", "i", "A", "z"))
    with pytest.raises(TypeError):
        ssa.ssm_glr_fwd(x.half(), r.half(), i.half(), A)
    with pytest.raises(TypeError):
        ssa.ssm_glr_fwd(x, r.bfloat16(), i, A)
    with pytest.raises(ValueError):
        ssa.ssm_glr_fwd(x, r, i)                                     # no A
    with pytest.raises(ValueError):
        ssa.ssm_glr_fwd(x, r, i, A, form="convex")
    with pytest.raises(KeyError):
        ssa.ssm_glr_fwd(x, r, i, A, form="other")
    with pytest.raises(ValueError):
        ssa.ssm_glr_fwd(x, r[:, :5], i, A)
    with pytest.raises(ValueError):
        ssa.ssm_glr_fwd(x, r.transpose(1, 2).contiguous().transpose(1, 2), i, A)    # channels apart
    with pytest.raises(ValueError):
        ssa.ssm_glr_fwd(x, torch.cat([r, r], 1)[:, ::2], i[:, :1].expand(1, 6, 8), A)  # rows on each other
    with pytest.raises(TypeError):
        ssa.ssm_glr_fwd(x, r, i, A, seqlens=torch.tensor([4]))       # int64
    with pytest.raises(ValueError):
        ssa.ssm_glr_fwd(x, r, i, A)                                  # not on a GPU
    with pytest.raises(ValueError):
        ssa.ssm_glr_step(t["h0"], x, r, i, A)                        # 3-D
    with pytest.raises(ValueError):
        ssa.ssm_add_norm_fwd(x, p=0.5)                               # no generator
    with pytest.raises(TypeError):
        ssa.ssm_add_norm_fwd(x, residual=x.half())
    with pytest.raises(ValueError):
        ssa.ssm_add_norm_fwd(x, weight=A[:4])
    with pytest.raises(KeyError):
        ssa.ssm_add_norm_fwd(x, norm="batch")
    with pytest.raises(TypeError):
        ssa.ssm_dropout(x, 0.5, torch.tensor([1.0, 2.0]))


def test_strided_rows_are_recognised():
    B, L, D = 2, 5, 8
    wide = torch.zeros((B, L, 3 * D))
    for k in range(3):
        v = wide[..., k * D:(k + 1) * D]
        assert ops._strided(v, "v", (B, L, D), torch.float32, v.device) == (v.data_ptr(), 3 * D)
    one = wide[:, 0, :D]  # a step's rows of a longer sequence
    assert ops._strided(one, "one", (B, D), torch.float32, one.device) == (one.data_ptr(), 3 * D * L)
    far = torch.empty_strided((2, 2), (2 ** 31, 1), device="meta")
    with pytest.raises(ValueError):
        ops._strided(far, "far", (2, 2), torch.float32, far.device)
    with pytest.raises(ValueError):
        ops._strided(wide[:, :3, :D], "cut", (B, 3, D), torch.float32, wide.device)  # batches not evenly after rows
    single = wide[:1, :3, :D]
    assert ops._strided(single, "single", (1, 3, D), torch.float32, wide.device)[1] == 3 * D
