"""Statistics of the group norm where one lane passes over thousands of positions, with a first
position far from all others (a border of zeros around data with an offset, one large first token):
digits lost to whatever the rows are compared with would show here."""
import pytest
import torch

import selective_scan_amd as ssa
from gpu_util import DEV

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
U = 2.0 ** -24


@pytest.mark.parametrize("first,offset", [(0.0, 100.0), (1000.0, 0.0), (None, 300.0)],
                         ids=["zero_border", "large_first", "offset"])
@pytest.mark.parametrize("S,C,G,dtype,rl", [(16384, 33, 1, F32, 7), (4096, 64, 8, F32, 16), (4096, 1024, 16, BF16, 2)],
                         ids=["33in1_f32", "64in8_f32", "1024in16_bf16"])
def test_statistics_over_many_positions(S, C, G, dtype, rl, first, offset):
    """385 samples are enough workgroups that none of them shares its positions (rl rows at once).
    The bound, with u = 2^-24, for squared distances formed in batches of eight rows and merged by
    count, mean and sum of squares. The sum of squares adds terms >= 0: relative u for each of the
    at most S / (8 rl) + 8 additions of a lane, rl of a channel, C / G / 64 + 64 of a group and its
    roundings. A batch's mean is off by e <= 4 u times its rows' root mean square, in either
    direction; what that adds to the sum, 2 sum 8 d e over the batches' distances d, is at most
    2 sqrt(sum 8 d^2) sqrt(sum 8 e^2) <= 8 u rms(x) / sigma of it. rstd takes half of the sum's
    error and 4 roundings of its own. The mean: additions of numbers no larger than |x|."""
    M = 385
    gen = torch.Generator(device=DEV).manual_seed(S + C)
    x = torch.randn((M, S, C), generator=gen, device=DEV, dtype=dtype)
    x += offset
    if first is not None:
        x[:, 0] = first
    y, mean, rstd = ssa.ssm_group_norm_fwd(x, G)
    torch.cuda.synchronize()
    cg = C // G
    adds = S / (8 * rl) + 8 + rl + cg / 64 + 64
    for m in (0, 200, M - 1):
        t = x[m].double().cpu().reshape(S, G, cg)
        want = t.mean(dim=(0, 2))
        var = ((t - want[:, None]) ** 2).mean(dim=(0, 2))
        r = 1 / torch.sqrt(var + 1e-5)
        rms = torch.sqrt((t ** 2).mean(dim=(0, 2)))
        off = (rstd[m].double().cpu() / r - 1).abs() / ((adds / 2 + 4) * U + 4 * U * rms * r)
        assert float(off.max()) <= 1.0, f"rstd of sample {m}: {float(off.max()):.2f} times the bound"
        off = (mean[m].double().cpu() - want).abs() / ((rl + cg / 64 + 64) * U * t.abs().mean(dim=(0, 2)))
        assert float(off.max()) <= 1.0, f"mean of sample {m}: {float(off.max()):.2f} times the bound"
        # y from the statistics that were returned: storage's rounding and three of its own
        xh = (t - mean[m].double().cpu()[:, None]) * rstd[m].double().cpu()[:, None]
        lim = torch.finfo(dtype).eps / 2 * xh.abs() + 4 * U * (t.abs() + want.abs()[:, None]) * r[:, None] + 1e-30
        assert bool(((y[m].double().cpu().reshape(S, G, cg) - xh).abs() <= 1.01 * lim).all()), f"y of sample {m}"


@pytest.mark.parametrize("M,S,C,G", [((1 << 22) + 5, 8, 32, 2), ((1 << 22) + 5, 9, 9, 3), (70000, 40, 64, 8),
                                     (3, 100001, 24, 4), ((1 << 22) + 5, 1, 64, 1)])
def test_sums_over_many_samples_are_exact(M, S, C, G):
    """dweight and dbias where the workgroups that add up their parts come behind more samples than one
    grid dimension takes, and on the ways beside it. Small whole numbers, statistics 0 and 1: every
    product and every partial sum (far below 2^24) is exact in 32 bits, and so are the results."""
    gen = torch.Generator(device=DEV).manual_seed(7)
    x, dy = (torch.randint(-2, 3, (M, S, C), generator=gen, device=DEV, dtype=torch.int8) for _ in range(2))
    mean, rstd = torch.zeros((M, G), device=DEV), torch.ones((M, G), device=DEV)
    g = ssa.ssm_group_norm_bwd(x.to(BF16), G, mean, rstd, dy.to(BF16))
    torch.cuda.synchronize()
    db, dw = (torch.zeros(C, dtype=torch.int64, device=DEV) for _ in range(2))
    for a in range(0, M, 1 << 18):
        p, q = x[a:a + (1 << 18)].reshape(-1, C), dy[a:a + (1 << 18)].reshape(-1, C)
        db += q.sum(0, dtype=torch.int64)
        dw += (p * q).sum(0, dtype=torch.int64)
    assert float(max(db.abs().max(), dw.abs().max())) < 2 ** 22
    assert torch.equal(g["dbias"].double(), db.double()) and torch.equal(g["dweight"].double(), dw.double())
