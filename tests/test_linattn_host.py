"""Linear attention and group norm without a GPU: the 64-bit forms the GPU tests use
against autograd and differences, and the refusals of the C ABI and of the binding
(all before any HIP call)."""
import ctypes

import pytest
import torch

import linattn_ref as ref
import selective_scan_amd as ssa
from selective_scan_amd import ops

P = ctypes.c_void_p(0x10000)
P2 = ctypes.c_void_p(0x20000)
ODD = ctypes.c_void_p(0x10004)


def _recurrence(q, k, v, a, scale, seqlens, h0):
    """Step by step, differentiable."""
    B, L, H, V = v.shape
    r = H // q.shape[2]
    q, k = q.repeat_interleave(r, 2), k.repeat_interleave(r, 2)
    S = h0
    lam = torch.exp(a)[None, :, None, None]
    out = []
    for t in range(L):
        live = torch.tensor([1.0 if t < n else 0.0 for n in ref._lens(seqlens, B, L)], dtype=torch.float64)
        live = live[:, None, None, None]
        S = live * (lam * S + k[:, t, :, :, None] * v[:, t, :, None, :]) + (1 - live) * S
        out.append(live[..., 0] * scale * (q[:, t, :, :, None] * S).sum(2))
    return torch.stack(out, 1), S


@pytest.mark.parametrize("G,seqlens", [(4, None), (2, [7, 0]), (1, [3, 9])])
def test_the_64_bit_forms_agree_with_the_recurrence_and_its_autograd(G, seqlens):
    B, L, H, K, V = 2, 9, 4, 5, 3
    t = ref.inputs(B, L, H, G, K, V, torch.float64, seed=1)
    a = t["log_decay"].double()
    x = {n: t[n].double().requires_grad_() for n in ("q", "k", "v", "h0")}
    o, S = _recurrence(x["q"], x["k"], x["v"], a, 0.3, seqlens, x["h0"])
    ro, rs = ref.fwd(t["q"], t["k"], t["v"], a, 0.3, seqlens, t["h0"].double())
    assert torch.allclose(o, ro, atol=1e-12) and torch.allclose(S, rs, atol=1e-12)
    l = (o * t["dout"].double()).sum() + (S * t["dh_final"].double()).sum()
    want = dict(zip(("dq", "dk", "dv", "dh0"), torch.autograd.grad(l, list(x.values()))))
    got = ref.bwd(t["q"], t["k"], t["v"], a, 0.3, t["dout"], seqlens, t["h0"].double(), t["dh_final"].double())
    for n in want:
        assert torch.allclose(got[n], want[n], atol=1e-11), n


@pytest.mark.parametrize("act", ["none", "silu"])
@pytest.mark.parametrize("gate", [False, True])
def test_the_64_bit_group_norm_gradient_is_autograds(act, gate):
    g = torch.Generator().manual_seed(3)
    r = lambda *s: torch.randn(s, generator=g, dtype=torch.float64)  # noqa: E731
    x, w, b, z, dy = r(2, 5, 12), r(12), r(12), r(2, 5, 12) if gate else None, r(2, 5, 12)
    leaves = [t.requires_grad_() for t in (x, w, b, z) if t is not None]
    y, mean, rstd = ref.norm_fwd(x, 3, w, b, z, act=act)
    want = torch.autograd.grad((y * dy).sum(), leaves)
    got = ref.norm_bwd(x, 3, mean, rstd, dy, w, b, z, act=act)
    for n, t in zip(("dx", "dweight", "dbias", "dz"), want):
        assert torch.allclose(got[n], t, atol=1e-11), n


def _fwd(B=2, L=8, H=4, G=2, K=64, V=128, io=1, q=P, k=P, v=P, a=P, scale=1.0, lens=None, h0=None, norm=None, o=P,
         hf=None, ws=P, wsb=1 << 40):
    return ops.lib().ssm_linattn_fwd(B, L, H, G, K, V, io, q, k, v, a, scale, lens, h0, norm, o, hf, ws, wsb, None)


def _norm(weight=None, bias=None, z=None, eps=1e-5):
    return ctypes.byref(ops._LinattnNorm(weight, bias, z, eps))


# every case has exactly one defect, so no call reaches a launch
DIMS = [(dict(B=0), 1), (dict(L=-1), 1), (dict(H=0), 1), (dict(G=0), 1), (dict(G=3), 1), (dict(io=4), 1),
        (dict(K=32), 2), (dict(V=96), 2), (dict(K=256), 2), (dict(B=70000), 2), (dict(H=65536, G=1), 2),
        (dict(B=65535, H=1024, G=1024), 2), (dict(L=(1 << 30) + 1, B=1, H=1, G=1), 2),
        (dict(B=4096, H=1025, G=1), 2)]


@pytest.mark.parametrize("kw,status", DIMS + [
    (dict(q=None), 1), (dict(k=None), 1), (dict(v=None), 1), (dict(a=None), 1), (dict(o=None), 1),
    (dict(q=ODD), 1), (dict(lens=ODD), 1), (dict(hf=ODD), 1), (dict(h0=P2, hf=P2), 1),
    (dict(norm=_norm(eps=0.0)), 1), (dict(norm=_norm(eps=float("nan"))), 1), (dict(norm=_norm(z=ODD)), 1),
    (dict(norm=_norm(), H=1024, G=1024), 2),
])
def test_linattn_fwd_rejects(kw, status):
    assert _fwd(**kw) == status
    assert ops.lib().ssm_last_error().startswith(b"ssm_linattn_fwd: ")


def _bwd(B=2, L=8, H=4, G=2, K=64, V=128, io=1, ws=P, wsb=1 << 40, **kw):
    a = dict(q=P, k=P, v=P, a=P, lens=None, h0=None, dout=P, T=None, dq=P, dk=P, dv=P, dh0=None)
    a.update(kw)
    return ops.lib().ssm_linattn_bwd(B, L, H, G, K, V, io, a["q"], a["k"], a["v"], a["a"], 1.0, a["lens"], a["h0"],
                                     a["dout"], a["T"], a["dq"], a["dk"], a["dv"], a["dh0"], ws, wsb, None)


@pytest.mark.parametrize("kw,status", DIMS + [
    (dict(dout=None), 1), (dict(dq=None), 1), (dict(dv=None), 1), (dict(a=None), 1), (dict(dk=ODD), 1),
    (dict(T=P2, dh0=P2), 1), (dict(ws=None, wsb=0), 3), (dict(wsb=64), 3),
])
def test_linattn_bwd_rejects(kw, status):
    assert _bwd(**kw) == status
    assert ops.lib().ssm_last_error().startswith(b"ssm_linattn_bwd: ")


@pytest.mark.parametrize("kw,status", [(c, s) for c, s in DIMS if "L" not in c] + [
    (dict(state=None), 1), (dict(q=None), 1), (dict(o=None), 1), (dict(state=ODD), 1), (dict(norm=_norm(eps=-1.0)), 1),
    (dict(norm=_norm(weight=ODD)), 1),
])
def test_linattn_step_rejects(kw, status):
    a = dict(B=2, H=4, G=2, K=64, V=128, io=1, state=P, q=P, k=P, v=P, a=P, norm=None, o=P)
    a.update(kw)
    assert ops.lib().ssm_linattn_step(a["B"], a["H"], a["G"], a["K"], a["V"], a["io"], a["state"], a["q"], a["k"],
                                      a["v"], a["a"], 1.0, a["norm"], a["o"], None) == status
    assert ops.lib().ssm_last_error().startswith(b"ssm_linattn_step: ")


NDIMS = [(dict(M=-1), 1), (dict(S=0), 1), (dict(C=0), 1), (dict(G=0), 1), (dict(G=5), 1), (dict(io=2), 1),
         (dict(act=2), 1), (dict(C=65600, G=1), 2), (dict(M=1 << 20, S=1 << 20), 2),
         (dict(M=1, S=(1 << 30) + 1, C=1, G=1), 2), (dict(M=1 << 21, S=1, C=1024, G=1024), 2)]


@pytest.mark.parametrize("kw,status", NDIMS + [
    (dict(eps=0.0), 1), (dict(x=None), 1), (dict(y=None), 1), (dict(mean=None), 1), (dict(x=ODD), 1), (dict(z=ODD), 1),
])
def test_group_norm_fwd_rejects(kw, status):
    a = dict(M=2, S=3, C=24, G=4, io=1, act=0, x=P, w=None, b=None, z=None, eps=1e-5, y=P, mean=P, rstd=P)
    a.update(kw)
    assert ops.lib().ssm_group_norm_fwd(a["M"], a["S"], a["C"], a["G"], a["io"], a["act"], a["x"], a["w"], a["b"],
                                        a["z"], a["eps"], a["y"], a["mean"], a["rstd"], P, 1 << 40, None) == status
    assert ops.lib().ssm_last_error().startswith(b"ssm_group_norm_fwd: ")


@pytest.mark.parametrize("kw,status", NDIMS + [
    (dict(x=None), 1), (dict(dy=None), 1), (dict(dx=None), 1), (dict(rstd=None), 1), (dict(z=P), 1), (dict(dz=P), 1),
    (dict(dw=ODD), 1),
])
def test_group_norm_bwd_rejects(kw, status):
    a = dict(M=2, S=3, C=24, G=4, io=1, act=0, x=P, w=None, b=None, z=None, mean=P, rstd=P, dy=P, dx=P, dw=P, db=P,
             dz=None)
    a.update(kw)
    assert ops.lib().ssm_group_norm_bwd(a["M"], a["S"], a["C"], a["G"], a["io"], a["act"], a["x"], a["w"], a["b"],
                                        a["z"], a["mean"], a["rstd"], a["dy"], a["dx"], a["dw"], a["db"], a["dz"], P,
                                        1 << 40, None) == status
    assert ops.lib().ssm_last_error().startswith(b"ssm_group_norm_bwd: ")


def _refused(status):
    assert status == 1
    assert b"an output must not be" in ops.lib().ssm_last_error()


def test_outputs_that_are_inputs_or_each_other_are_refused():
    L, n = ops.lib(), [0x10000 * (i + 1) for i in range(16)]
    dims = (2, 8, 2, 2, 64, 64, 1)
    for o, hf, h0, z in ((n[2], None, None, None), (n[0], None, None, None), (n[4], n[5], n[5], None),
                         (n[4], n[4], None, None), (n[4], None, None, n[4])):
        _refused(L.ssm_linattn_fwd(*dims, *n[:4], 1.0, None, h0, _norm(z=z) if z else None, o, hf, n[9], 1 << 40, None))
    for at in range(4):
        outs = n[8:12]
        for other in (n[0], n[5], outs[(at + 1) % 4]):
            _refused(L.ssm_linattn_bwd(*dims, *n[:4], 1.0, None, None, n[4], n[5],
                                       *(other if i == at else x for i, x in enumerate(outs)), n[15], 1 << 40, None))
    for o, z in ((n[3], None), (n[0], None), (n[6], n[6])):
        _refused(L.ssm_linattn_step(2, 2, 2, 64, 64, 1, n[0], n[1], n[2], n[3], n[4], 1.0, _norm(z=z), o, None))
    for y, mean, rstd in ((n[3], n[5], n[6]), (n[4], n[5], n[5]), (n[4], n[0], n[6]), (n[4], n[4], n[6])):
        _refused(L.ssm_group_norm_fwd(2, 3, 24, 4, 1, 0, n[0], n[1], n[2], n[3], 1e-5, y, mean, rstd, n[9], 1 << 40, None))
    for at in range(4):
        outs = n[8:12]
        for other in (n[0], n[6], outs[(at + 1) % 4]):
            _refused(L.ssm_group_norm_bwd(2, 3, 24, 4, 1, 0, *n[:7],
                                          *(other if i == at else x for i, x in enumerate(outs)), n[15], 1 << 40, None))


def test_workspace_sizes_of_refused_shapes_are_zero():
    assert ssa.ssm_linattn_workspace_size(1, 4096, 16, 16, 96, 128) == 0
    assert ssa.ssm_linattn_bwd_workspace_size(1, 4096, 16, 5, 128, 128) == 0
    assert ssa.ssm_group_norm_workspace_size(4, 4096, 320, 7) == 0
    assert ssa.ssm_linattn_bwd_workspace_size(1, 4096, 16, 4, 128, 128) > 0


def test_the_binding_checks_its_tensors():
    t = ref.inputs(1, 4, 2, 2, 64, 64, torch.float32, seed=0)
    q, k, v, a = (t[n] for n in ("q", "k", "v", "log_decay"))
    with pytest.raises(TypeError):
        ssa.ssm_linattn_fwd(q.half(), k.half(), v.half(), a)
    with pytest.raises(TypeError):
        ssa.ssm_linattn_fwd(q, k, v.bfloat16(), a)
    with pytest.raises(ValueError):
        ssa.ssm_linattn_fwd(q, k[:, :3], v, a)
    with pytest.raises(ValueError):
        ssa.ssm_linattn_fwd(q, k.transpose(1, 2).contiguous().transpose(1, 2), v, a)
    with pytest.raises(TypeError):
        ssa.ssm_linattn_fwd(q, k, v, a, seqlens=torch.tensor([4]))          # int64
    with pytest.raises(ValueError):
        ssa.ssm_linattn_fwd(q, k, v, a, z=v)                                # a gate without norm_eps
    with pytest.raises(ValueError):
        ssa.ssm_group_norm_fwd(q, 2)                                        # 4-D
    with pytest.raises(KeyError):
        ssa.ssm_group_norm_fwd(q.reshape(4, 128), 2, act="gelu")
