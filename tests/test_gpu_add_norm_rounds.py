"""Residual add with norm, its gradient and dropout over so many rows that every workgroup walks
several: three rounds at least of each kind of row (16 lanes; a wave; several waves with several
rows a workgroup, or one; two octets a lane), every row against the 64-bit definitions and bounds
of test_gpu_add_norm.py. And the missing weight and bias. The masks are drawn by whole-tensor
arithmetic, which is held to the generator in Python's whole numbers."""
import pytest
import torch

import glr_ref as ref
import selective_scan_amd as ssa
import test_gpu_add_norm as base
from gpu_util import DEV

F32, BF16 = torch.float32, torch.bfloat16


def bits(seed, offset, M, C):
    """``ref.bits`` for many rows at once: 64-bit products from 32-bit words, of which a
    wrapped-around int64 keeps the right low bits and, shifted and masked, the right high ones."""
    n, m = -(-C // 8), 0xFFFFFFFF
    at = torch.arange(M * n) + (offset % 2 ** 64 - (2 ** 64 if offset % 2 ** 64 >= 2 ** 63 else 0))
    c = [at & m, (at >> 32) & m, torch.zeros_like(at), torch.zeros_like(at)]
    k = [seed & m, (seed >> 32) & m]
    for _ in range(10):
        p0, p1 = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
        c = [((p1 >> 32) & m) ^ c[1] ^ k[0], p1 & m, ((p0 >> 32) & m) ^ c[3] ^ k[1], p0 & m]
        k = [(k[0] + 0x9E3779B9) & m, (k[1] + 0xBB67AE85) & m]
    halves = torch.stack([h for w in c for h in (w & 0xFFFF, w >> 16)], 1)
    return halves.reshape(M, n * 8)[:, :C]


@pytest.mark.parametrize("rng", [base.RNG, (0, 0), (-3, 2 ** 63 - 2), (2 ** 63 - 1, -5)])
def test_masks_of_many_rows_are_the_generators(rng):
    for M, C in ((1, 1), (3, 8), (7, 21)):
        assert torch.equal(bits(*rng, M, C), ref.bits(*rng, M, C))


# rows, channels: the rows of one round are 12288, 3072, 1536, 1024, and 256 from there on
MANY = [(40000, 9), (37001, 128), (10000, 136), (9500, 512), (5000, 520), (3500, 1536), (800, 5000), (790, 8192),
        (780, 9001), (770, 12500)]


@pytest.mark.gpu
@pytest.mark.parametrize("types", [(BF16, F32), (F32, F32), (BF16, BF16)], ids=str)
@pytest.mark.parametrize("shape", MANY, ids=lambda s: "x".join(map(str, s)))
def test_every_row_of_three_rounds(shape, types, monkeypatch):
    monkeypatch.setattr(ref, "bits", bits)
    norm, p = [("layer", 0.1), ("rms", 0.0), ("rms", 0.3)][(shape[1] + (types[0] is F32) + 2 * (types[1] is BF16)) % 3]
    base.check(base.make(*shape, *types, seed=sum(shape)), norm, p, what=f"{shape} {norm} {p} {types}")


@pytest.mark.gpu
@pytest.mark.parametrize("shape", [(40000, 9), (10000, 136), (3500, 1536), (780, 9001)], ids=str)
def test_layer_norm_with_dropout_of_many_rows(shape, monkeypatch):
    monkeypatch.setattr(ref, "bits", bits)
    base.check(base.make(*shape, BF16, F32, seed=1 + sum(shape)), "layer", 0.2, what=f"{shape}")


@pytest.mark.gpu
@pytest.mark.parametrize("norm", ["layer", "rms"])
@pytest.mark.parametrize("shape", [(5, 7), (13001, 96), (6, 300), (3500, 1001), (3, 9001)], ids=str)
def test_no_weight_and_no_bias_are_ones_and_zeros(shape, norm):
    """With a weight of ones and a bias of zeros to the 64-bit bounds; without them the same bits."""
    t = base.make(*shape, BF16, F32, seed=7)
    t["w"], t["b"] = torch.ones_like(t["w"]), torch.zeros_like(t["b"])
    base.check(t, norm, 0.0, what=f"{shape} {norm}")
    d = {k: v.to(DEV) for k, v in t.items()}
    want = ssa.ssm_add_norm_fwd(d["x"], d["residual"], d["w"], d["b"], norm=norm)
    for w, b in ((None, None), (d["w"], None), (None, d["b"])):
        got = ssa.ssm_add_norm_fwd(d["x"], d["residual"], w, b, norm=norm)
        torch.cuda.synchronize()
        assert all(u is v is None or torch.equal(u, v) for u, v in zip(want, got))
    g = ssa.ssm_add_norm_bwd(*want[1:], d["dy"], d["w"], d["dsum"], norm=norm)
    g2 = ssa.ssm_add_norm_bwd(*want[1:], d["dy"], None, d["dsum"], norm=norm)
    torch.cuda.synchronize()
    assert all(torch.equal(g[n], g2[n]) for n in g)


@pytest.mark.gpu
@pytest.mark.parametrize("shape", [(40000, 9), (10000, 136), (5000, 520), (3500, 1536), (780, 9001)], ids=str)
def test_in_place_over_many_rows(shape):
    """The next row's loads are under way while the present one is written."""
    t = base.make(*shape, BF16, F32, seed=8)
    d = {k: v.to(DEV) for k, v in t.items()}
    kw = dict(p=0.2, rng=base.rng_tensor())
    y, s, mean, rstd = ssa.ssm_add_norm_fwd(d["x"], d["residual"], d["w"], d["b"], **kw)
    g = ssa.ssm_add_norm_bwd(s, mean, rstd, d["dy"], d["w"], d["dsum"], **kw)
    x, res, ds, z = d["x"].clone(), d["residual"].clone(), d["dsum"].clone(), d["x"].clone()
    ssa.ssm_add_norm_fwd(x, res, d["w"], d["b"], y=x, sum=res, **kw)
    g2 = ssa.ssm_add_norm_bwd(s, mean, rstd, d["dy"], d["w"], ds, out=dict(dresidual=ds), **kw)
    ssa.ssm_dropout(z, y=z, **kw)
    torch.cuda.synchronize()
    assert torch.equal(x, y) and torch.equal(res, s) and torch.equal(ds, g["dresidual"])
    assert all(torch.equal(g[n], g2[n]) for n in g) and torch.equal(z, ssa.ssm_dropout(d["x"], **kw))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_dropout_of_more_octets_than_one_round_takes(dtype):
    """2^21 octets are under way at once; these are 2.5 times as many, the last of a row not whole."""
    M, C, p = 40000, 1045, 0.1
    x = torch.randn((M, C), generator=torch.Generator().manual_seed(3)).to(dtype)
    y = ssa.ssm_dropout(x.to(DEV), p, base.rng_tensor()).cpu()
    for at in range(0, M, 5000):
        n = -(-C // 8)
        least = round(65536 * p)
        f = (bits(base.RNG[0], base.RNG[1] + at * n, 5000, C) >= least).double() * (65536 / (65536 - least))
        v = x[at:at + 5000].double()
        ref.close(y[at:at + 5000], v * f, v.abs() * 2.0 ** -24, 1.0, f"rows from {at}", store=dtype)
