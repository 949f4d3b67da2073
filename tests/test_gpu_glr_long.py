"""Gated linear recurrence, residual add with norm, and dropout on tensors of more than 2^31
elements: rows at both ends against 64 bits. The recurrence's gates are half open there, so that a
step's result depends on some hundred steps around it (a decay of at most 0.99 a step at the gates'
five deviations, a half at the middle: over 3000 steps nothing of fp32's precision is left)."""
import pytest
import torch

import glr_ref as ref
import selective_scan_amd as ssa
from gpu_util import DEV

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


def normal(shape, seed, dtype=BF16):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return torch.randn(shape, generator=g, device=DEV, dtype=dtype)


def test_a_recurrence_over_more_than_2_31_elements():
    B, L, D, n = 2, 1 << 20, 1032, 3200
    shape = (B, L, D)
    assert B * L * D > 2 ** 31
    print("inputs", flush=True)
    x, r, dy = (normal(shape, s) for s in range(3))
    pick = torch.tensor([0, 1, 63, 64, 1000, 1031], device=DEV)
    cut = lambda t, at: t[:, at:at + n, :][..., pick].cpu()  # noqa: E731
    print("forward", flush=True)
    y, h, states = ssa.ssm_glr_fwd(x, r, form="convex", want_states=True)
    torch.cuda.synchronize()
    out = None
    for at in (0, L - n):
        t = dict(x=cut(x, at), r=cut(r, at), dy=cut(dy, at),
                 h0=None if at == 0 else states[:, at // 128][:, pick].cpu())
        g = ref.Glr(t, "convex", None, t["dy"])
        ref.close(cut(y, at), g.y, g.ey, 1.0, f"y at {at}", store=BF16)
        if at:
            ref.close(h[:, pick].cpu(), g.h_final, g.eh_final, 1.0, "h_final", store=F32)
        if out is None:
            print("gradient", flush=True)
            out = ssa.ssm_glr_bwd(x, r, states, dy, form="convex")
            torch.cuda.synchronize()
        for k in ("dx", "dr"):
            v, e = g.out[k]
            got = cut(out[k], at)
            if at == 0:  # without the last steps of the piece, whose gradient comes from behind it
                got, v, e = got[:, :n - 3000 + 128], v[:, :n - 3000 + 128], e[:, :n - 3000 + 128]
            ref.close(got, v, e, 1.0, f"{k} at {at}", store=BF16)


def test_norms_and_dropout_over_more_than_2_31_elements():
    M, C = 265000, 8200
    assert M * C > 2 ** 31
    print("inputs", flush=True)
    x, res = normal((M, C), 3), normal((M, C), 4)
    w = 1 + 0.1 * normal((C,), 5, F32)
    rng = torch.tensor([7, 11], dtype=torch.int64, device=DEV)
    n = -(-C // 8)
    print("forward", flush=True)
    y, s, mean, rstd = ssa.ssm_add_norm_fwd(x, res, w, p=0.2, rng=rng)
    torch.cuda.synchronize()
    rows = [0, 1, M // 2, M - 2, M - 1]
    f = torch.cat([ref.factor(0.2, (7, 11 + m * n), 1, C) for m in rows])
    at = lambda t: t[rows].cpu()  # noqa: E731
    ry, rs, rm, rr = ref.add_norm_fwd(at(x), at(res), w.cpu(), None, 1e-5, "layer", f)
    # sums of 8200 terms of order one: relative 2^-15 holds with room (test_gpu_add_norm.py has the bounds)
    ref.close(at(y), ry, ry.abs() + 1, 2.0 ** -15, "y", store=BF16)
    ref.close(at(s), rs, rs.abs() + 1, 2.0 ** -20, "sum", store=BF16)
    print("gradient", flush=True)
    g = ssa.ssm_add_norm_bwd(s, mean, rstd, x, w, res, p=0.2, rng=rng, out=dict(dresidual=y))
    torch.cuda.synchronize()
    r = ref.add_norm_bwd(at(s), at(mean), at(rstd), at(x), w.cpu(), at(res), "layer", f)
    ref.close(at(g["dresidual"]), r["dresidual"], r["dresidual"].abs() + 1, 2.0 ** -15, "dresidual", store=BF16)
    ref.close(at(g["dx"]), r["dx"], (r["dresidual"].abs() + 1) * 1.25, 2.0 ** -15, "dx", store=BF16)
    del y, g
    print("dropout", flush=True)
    z = ssa.ssm_dropout(x, 0.2, rng, y=s)
    torch.cuda.synchronize()
    ref.close(at(z), at(x).double() * f, at(x).double().abs(), 2.0 ** -23, "dropout", store=BF16)
