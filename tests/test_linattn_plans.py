"""Linear attention on sequences cut every way the library cuts them: super-chunks of many chunks, what
they add to the state in one piece or several, two or three heads of a group in one workgroup, lengths
that end inside each of these. The plan of every case is asserted (no GPU needed), so that other plans
for these sizes would show as cases to be chosen anew; the results are held to the 64-bit definition."""
import pytest
import torch

import linattn_ref as ref
import selective_scan_amd as ssa

F32, BF16 = torch.float32, torch.bfloat16
DEV = "cuda:0"

# B, L, H, G, K, V, dtype, lengths; super-chunks, chunks of one, pieces, heads together
FWD = [
    ((4, 8000, 24, 8, 128, 64), BF16, [8000, 2500, 1650, 6111], (5, 25, 2, 1)),
    ((4, 8000, 24, 8, 64, 128), BF16, None, (5, 25, 2, 1)),
    ((2, 9000, 40, 40, 128, 128), BF16, [5000, 8999], (3, 47, 4, 1)),
    ((3, 5000, 32, 32, 64, 64), F32, [0, 1025, 4999], (5, 16, 2, 1)),
    ((4, 2047, 24, 8, 128, 64), F32, [2047, 1000, 513, 1024], (2, 16, 2, 1)),
    ((4, 2047, 24, 8, 64, 64), BF16, [1, 2047, 300, 1500], (8, 4, 1, 1)),
    ((1, 12000, 8, 8, 128, 128), BF16, [11111], (32, 6, 1, 1)),
]
BWD = [
    ((4, 2047, 24, 8, 128, 64), BF16, [2047, 1000, 513, 1111], (4, 8, 1, 3)),
    ((4, 2047, 24, 8, 64, 64), BF16, [300, 2047, 1, 1666], (8, 4, 1, 3)),
    ((4, 5000, 48, 16, 128, 64), BF16, [5000, 1300, 3900, 2561], (2, 40, 2, 3)),
    ((1, 4096, 24, 12, 128, 64), BF16, [3000], (10, 7, 1, 2)),
    ((2, 6000, 24, 24, 64, 64), BF16, [6000, 1900], (5, 19, 2, 1)),
    ((2, 6000, 24, 24, 64, 128), BF16, [640, 5555], (5, 19, 2, 1)),
    ((2, 6000, 24, 24, 128, 64), BF16, None, (5, 19, 2, 1)),
    ((2, 6000, 24, 24, 128, 128), BF16, [5999, 2600], (3, 32, 4, 1)),
    ((2, 6000, 24, 24, 128, 128), F32, [1217, 6000], (5, 19, 2, 1)),
    ((2, 3000, 24, 8, 128, 128), BF16, [2999, 1100], (3, 16, 2, 1)),
    ((2, 3000, 24, 8, 64, 64), F32, [3000, 1500], (3, 16, 2, 1)),
]
ALL = [(*c, 0) for c in FWD] + [(*c, 1) for c in BWD]


def names(cases):
    return [f"{'x'.join(map(str, c[0]))}_{'bf16' if c[1] == BF16 else 'f32'}" + ("_gradient" if c[-1] == 1 else "")
            for c in cases]


@pytest.mark.parametrize("shape,dtype,lens,plan,gradient", ALL, ids=names(ALL))
def test_plan(shape, dtype, lens, plan, gradient):
    io = 1 if dtype == BF16 else 0
    p = ssa.ssm_diag_linattn_plan(*shape, io, gradient)
    assert (p["supers"], p["per_super"], p["pieces"], p["together"]) == plan
    assert p["chunks"] == (shape[1] + 63) // 64 and p["per_piece"] * p["pieces"] >= p["per_super"]
    B, L, H, G, K, V = shape
    slots = B * H * K * V * 4 * (p["supers"] - 1) * p["pieces"]
    planes = 0 if H == G or p["together"] > 1 else 2 * B * L * H * K * 4
    need = ssa.ssm_linattn_bwd_workspace_size(*shape, io) if gradient else ssa.ssm_linattn_workspace_size(*shape, io)
    assert need == (2 * slots + planes if gradient else slots)


def test_plan_refuses_what_the_calls_refuse():
    with pytest.raises(ssa.SsmError):
        ssa.ssm_diag_linattn_plan(1, 100, 4, 3, 64, 64)
    with pytest.raises(ssa.SsmError):
        ssa.ssm_diag_linattn_plan(1, 100, 4, 4, 96, 64)


def check(got, want, mag, c, what):
    """Every value within its bound, and the 2-norm per (batch, head): a rounding of the output is at
    most half a step of each value, hence of the norm; what the products lose (2^-18 of each for a pair of
    bf16 numbers, three of these on the way; a few 2^-24 in 32 bits, as many as sixteen independent ones)
    is of either sign. A state that is carried wrongly changes the norm by far more."""
    ref.close(got, want.cpu(), mag.cpu(), c, what)
    heads = 2 if what.startswith("d") and what[1] in "qkv" or what == "o" else 1
    dims = (1, 3) if heads == 2 else (2, 3)
    lost = {BF16: 2.0 ** -8 + 2.0 ** -15, F32: 32 * 2.0 ** -24}[got.dtype]
    off = (got.double() - want).square().sum(dims).sqrt()
    assert bool((off <= lost * want.square().sum(dims).sqrt() + 1e-30).all()), f"{what}: norm"


def prepared(shape, dtype, lens, seed):
    """(inputs with padding that is not finite, the same with zeros there), on the GPU."""
    t = ref.inputs(*shape, dtype, seed=seed, device=DEV)
    clean = dict(t)
    if lens is not None:
        for n in ("q", "k", "v", "dout"):
            clean[n] = t[n].clone()
            for b, m in enumerate(lens):
                clean[n][b, m:] = 0
                t[n][b, m:] = float("nan")
    seqlens = None if lens is None else torch.tensor(lens, dtype=torch.int32, device=DEV)
    return t, clean, seqlens


@pytest.mark.gpu
@pytest.mark.parametrize("shape,dtype,lens,plan", FWD, ids=names(FWD))
def test_forward(shape, dtype, lens, plan):
    B, L, H, G, K, V = shape
    t, u, seqlens = prepared(shape, dtype, lens, L)
    o, hf = ssa.ssm_linattn_fwd(t["q"], t["k"], t["v"], t["log_decay"], seqlens=seqlens, h0=t["h0"])
    torch.cuda.synchronize()
    args = (u["q"], u["k"], u["v"], u["log_decay"], K ** -0.5)
    with torch.device(DEV):
        ro, rh = ref.fwd(*args, seqlens=lens, h0=u["h0"])
        mo, mh = ref.magnitude(ref.fwd, *args, seqlens=lens, h0=u["h0"])
    c = ref.term_error(L, K, V, dtype == BF16)
    check(o, ro, mo, c, "o")
    check(hf, rh, mh, c, "h_final")
    for b, n in enumerate(lens or []):
        assert not o[b, n:].any()


@pytest.mark.gpu
@pytest.mark.parametrize("shape,dtype,lens,plan", BWD, ids=names(BWD))
def test_gradient(shape, dtype, lens, plan):
    B, L, H, G, K, V = shape
    t, u, seqlens = prepared(shape, dtype, lens, L + 1)
    g = ssa.ssm_linattn_bwd(t["q"], t["k"], t["v"], t["log_decay"], t["dout"], seqlens=seqlens, h0=t["h0"],
                            dh_final=t["dh_final"])
    torch.cuda.synchronize()
    args = (u["q"], u["k"], u["v"], u["log_decay"], K ** -0.5, u["dout"])
    with torch.device(DEV):
        r = ref.bwd(*args, seqlens=lens, h0=u["h0"], T=u["dh_final"])
        m = ref.magnitude(ref.bwd, *args, seqlens=lens, h0=u["h0"], T=u["dh_final"])
    c = ref.term_error(L, K, V, dtype == BF16, extra=H // G)
    for n in ("dq", "dk", "dv", "dh0"):
        check(g[n], r[n], m[n], c, n)
    for b, n in enumerate(lens or []):
        assert not g["dq"][b, n:].any() and not g["dk"][b, n:].any() and not g["dv"][b, n:].any()
