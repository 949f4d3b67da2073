"""Linear attention with a decay per head on the GPU against its 64-bit definition:
forward, gradient and decode step, over types, head groups, lengths from 0 to a few
thousand, padding, decays from none to total, and the ways a program calls them."""
import pytest
import torch

import linattn_ref as ref
import selective_scan_amd as ssa
from gpu_util import DEV

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


def dev(t):
    return {n: (x.to(DEV) if torch.is_tensor(x) else x) for n, x in t.items()}


def lens_arg(seqlens):
    return None if seqlens is None else torch.tensor(seqlens, dtype=torch.int32, device=DEV)


def check_fwd(t, K, V, seqlens=None, scale=None, what=""):
    scale = K ** -0.5 if scale is None else scale
    d = dev(t)
    o, hf = ssa.ssm_linattn_fwd(d["q"], d["k"], d["v"], d["log_decay"], scale=scale, seqlens=lens_arg(seqlens),
                                h0=d["h0"])
    torch.cuda.synchronize()
    args = (t["q"], t["k"], t["v"], t["log_decay"], scale)
    ro, rh = ref.fwd(*args, seqlens=seqlens, h0=t["h0"])
    mo, mh = ref.magnitude(ref.fwd, *args, seqlens=seqlens, h0=t["h0"])
    c = ref.term_error(t["q"].shape[1], K, V, t["q"].dtype == BF16)
    ref.close(o, ro, mo, c, what + " o")
    ref.close(hf, rh, mh, c, what + " h_final")
    return o, hf


def check_bwd(t, K, V, seqlens=None, what="", **kw):
    scale = K ** -0.5
    d = dev(t)
    g = ssa.ssm_linattn_bwd(d["q"], d["k"], d["v"], d["log_decay"], d["dout"], scale=scale, seqlens=lens_arg(seqlens),
                            h0=d["h0"], dh_final=d["dh_final"], **kw)
    torch.cuda.synchronize()
    args = (t["q"], t["k"], t["v"], t["log_decay"], scale, t["dout"])
    r = ref.bwd(*args, seqlens=seqlens, h0=t["h0"], T=t["dh_final"])
    m = ref.magnitude(ref.bwd, *args, seqlens=seqlens, h0=t["h0"], T=t["dh_final"])
    heads = t["v"].shape[2] // t["q"].shape[2]
    c = ref.term_error(t["q"].shape[1], K, V, t["q"].dtype == BF16, extra=heads)
    for n in ("dq", "dk", "dv", "dh0"):
        if g[n] is not None:
            ref.close(g[n], r[n], m[n], c, f"{what} {n}")
    return g


SHAPES = [
    # B, L, H, G, K, V
    (1, 1, 1, 1, 64, 64), (2, 2, 2, 1, 128, 64), (1, 31, 2, 2, 64, 128), (2, 63, 3, 1, 128, 128),
    (1, 64, 2, 2, 128, 128), (1, 65, 4, 2, 64, 64), (3, 127, 2, 2, 128, 128), (1, 128, 3, 3, 64, 128),
    (2, 129, 6, 2, 128, 64), (1, 700, 5, 5, 128, 128), (2, 1500, 2, 1, 64, 64), (1, 2500, 1, 1, 128, 128),
    (5, 257, 7, 7, 64, 64), (2, 300, 3, 1, 64, 64), (1, 1300, 6, 2, 128, 64), (3, 70, 8, 2, 64, 64),
]


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_forward(shape, dtype):
    B, L, H, G, K, V = shape
    check_fwd(ref.inputs(*shape, dtype, seed=L, h0=L % 2 == 1), K, V, what=str(shape))


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_gradient(shape, dtype):
    B, L, H, G, K, V = shape
    check_bwd(ref.inputs(*shape, dtype, seed=L + 1, h0=L % 2 == 1), K, V, what=str(shape))


@pytest.mark.parametrize("decay", [0.0, -1e-6, -0.01, -1.0, -30.0, -1e6, float("-inf")])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_decays_from_none_to_total(decay, dtype):
    t = ref.inputs(1, 330, 2, 2, 64, 128, dtype, seed=5, decay=decay)
    check_fwd(t, 64, 128, what=f"decay {decay}")
    check_bwd(t, 64, 128, what=f"decay {decay}")


LENS = [[0, 1, 200], [200, 64, 65], [63, 128, 199], [-3, 1000, 0]]


@pytest.mark.parametrize("seqlens", LENS, ids=str)
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_padded_batches(seqlens, dtype):
    """Padding rows hold NaN and infinities: they reach no output, and their own outputs are 0."""
    B, L, H, G, K, V = 3, 200, 4, 2, 128, 64
    t = ref.inputs(B, L, H, G, K, V, dtype, seed=7)
    clean = {n: (x.clone() if x is not None else None) for n, x in t.items()}
    for b, n in enumerate(ref._lens(seqlens, B, L)):
        for name, bad in (("q", float("nan")), ("k", float("inf")), ("v", float("nan")), ("dout", float("-inf"))):
            t[name][b, n:] = bad
            clean[name][b, n:] = 0
    scale = K ** -0.5
    d = dev(t)
    args = (clean["q"], clean["k"], clean["v"], clean["log_decay"], scale)
    o, hf = ssa.ssm_linattn_fwd(d["q"], d["k"], d["v"], d["log_decay"], scale=scale, seqlens=lens_arg(seqlens),
                                h0=d["h0"])
    g = ssa.ssm_linattn_bwd(d["q"], d["k"], d["v"], d["log_decay"], d["dout"], scale=scale, seqlens=lens_arg(seqlens),
                            h0=d["h0"], dh_final=d["dh_final"])
    torch.cuda.synchronize()
    c = ref.term_error(L, K, V, dtype == BF16, extra=2)
    kw = dict(seqlens=seqlens, h0=t["h0"])
    ro, rh = ref.fwd(*args, **kw)
    mo, mh = ref.magnitude(ref.fwd, *args, **kw)
    ref.close(o, ro, mo, c, "o")
    ref.close(hf, rh, mh, c, "h_final")
    r = ref.bwd(*args, clean["dout"], T=t["dh_final"], **kw)
    m = ref.magnitude(ref.bwd, *args, clean["dout"], T=t["dh_final"], **kw)
    for n in r:
        ref.close(g[n], r[n], m[n], c, n)
    for b, n in enumerate(ref._lens(seqlens, B, L)):
        for x in (o, g["dq"], g["dk"], g["dv"]):
            assert not x[b, n:].any()


@pytest.mark.parametrize("B,H,L", [(1, 40, 300), (3, 100, 150), (2, 3, 4000)])
def test_more_heads_and_more_chunks_than_one_launch_wave(B, H, L):
    t = ref.inputs(B, L, H, H, 64, 64, BF16, seed=9, h0=True)
    check_fwd(t, 64, 64)
    check_bwd(t, 64, 64)


def test_values_outside_the_half_range():
    """Factors far from 1 (bf16 has fp32's range): nothing overflows or is flushed on the way."""
    t = ref.inputs(1, 200, 2, 2, 128, 128, BF16, seed=11)
    for big, small in ((2.0 ** 40, 2.0 ** -40), (2.0 ** -30, 2.0 ** 20)):
        u = dict(t, q=(t["q"].float() * big).to(BF16), k=(t["k"].float() * small).to(BF16), h0=None, dh_final=None)
        check_fwd(u, 128, 128, what=f"{big}")
        check_bwd(u, 128, 128, what=f"{big}")


def test_a_sequence_in_two_parts_and_then_token_by_token():
    """Prefill, prefill from its state, then steps: what one call over everything gives."""
    B, L, H, G, K, V = 2, 180, 4, 2, 64, 128
    t = ref.inputs(B, L, H, G, K, V, BF16, seed=13)
    d = dev(t)
    part = lambda a, b: [d[n][:, a:b].contiguous() for n in ("q", "k", "v")]  # noqa: E731
    o1, s1 = ssa.ssm_linattn_fwd(*part(0, 100), d["log_decay"], h0=d["h0"])
    o2, s2 = ssa.ssm_linattn_fwd(*part(100, 170), d["log_decay"], h0=s1)
    rows = [o1, o2]
    state = s2.clone()
    for i in range(170, L):
        q, k, v = (x[:, 0].contiguous() for x in part(i, i + 1))
        rows.append(ssa.ssm_linattn_step(state, q, k, v, d["log_decay"])[:, None])
    o = torch.cat(rows, 1)
    args = (t["q"], t["k"], t["v"], t["log_decay"], K ** -0.5)
    ro, rh = ref.fwd(*args, h0=t["h0"])
    mo, mh = ref.magnitude(ref.fwd, *args, h0=t["h0"])
    c = ref.term_error(L, K, V, True, pairs=6)
    ref.close(o, ro, mo, c, "o")
    ref.close(state, rh, mh, c, "state")


def test_length_zero():
    t = dev(ref.inputs(2, 0, 4, 2, 64, 64, BF16, seed=1))
    o, hf = ssa.ssm_linattn_fwd(t["q"], t["k"], t["v"], t["log_decay"], h0=t["h0"])
    assert o.shape == (2, 0, 4, 64) and torch.equal(hf, t["h0"])
    _, hf = ssa.ssm_linattn_fwd(t["q"], t["k"], t["v"], t["log_decay"])
    assert not hf.any()
    g = ssa.ssm_linattn_bwd(t["q"], t["k"], t["v"], t["log_decay"], t["dout"], h0=t["h0"], dh_final=t["dh_final"])
    assert torch.equal(g["dh0"], t["dh_final"])


@pytest.mark.parametrize("L", [150, 3000])
def test_optional_outputs(L):
    """Without the final state, or dh0, the others stay what they are (the state is then formed with
    fewer parts: the same bounds, not the same bits)."""
    B, H, G, K, V = 1, 2, 2, 64, 64
    t = ref.inputs(B, L, H, G, K, V, BF16, seed=3)
    d = dev(t)
    o, none = ssa.ssm_linattn_fwd(d["q"], d["k"], d["v"], d["log_decay"], h0=d["h0"], want_final_state=False)
    args = (t["q"], t["k"], t["v"], t["log_decay"], K ** -0.5)
    c = ref.term_error(L, K, V, True)
    assert none is None
    ref.close(o, ref.fwd(*args, h0=t["h0"])[0], ref.magnitude(ref.fwd, *args, h0=t["h0"])[0], c, "o")
    g = check_bwd(t, K, V, what="without dh0", want_dh0=False)
    assert g["dh0"] is None


def test_the_state_is_good_to_single_precision():
    """The state's products enter it in three bf16 parts (24 bits): the final state and dh0 are within a
    few fp32 roundings of the 64-bit ones, in the 2-norm."""
    B, L, H, G, K, V = 2, 2000, 4, 2, 128, 64
    t = ref.inputs(B, L, H, G, K, V, BF16, seed=51)
    d = dev(t)
    _, hf = ssa.ssm_linattn_fwd(d["q"], d["k"], d["v"], d["log_decay"], h0=d["h0"])
    g = ssa.ssm_linattn_bwd(d["q"], d["k"], d["v"], d["log_decay"], d["dout"], h0=d["h0"], dh_final=d["dh_final"])
    args = (t["q"], t["k"], t["v"], t["log_decay"], K ** -0.5)
    for got, want in ((hf, ref.fwd(*args, h0=t["h0"])[1]),
                      (g["dh0"], ref.bwd(*args, t["dout"], h0=t["h0"], T=t["dh_final"])["dh0"])):
        # each of the sum's roundings (at most L / 16 + a few, 2^-24 of a partial sum no larger than the
        # sum of absolute values) adds independently: 16 of them in the norm is beyond what they reach
        assert float((got.double().cpu() - want).norm() / want.norm()) < 16 * 2.0 ** -24


def test_gradient_against_differences_of_the_forward():
    """The operator is linear in each of q, k, v, h0, so a central difference of any width is exact
    up to rounding: <grad, d> = (l(x + d) - l(x - d)) / 2, with l summed in 64 bits."""
    B, L, H, G, K, V = 1, 150, 4, 2, 64, 64
    t = ref.inputs(B, L, H, G, K, V, F32, seed=17)
    d = dev(t)
    g = ssa.ssm_linattn_bwd(d["q"], d["k"], d["v"], d["log_decay"], d["dout"], h0=d["h0"], dh_final=d["dh_final"])

    def loss(**kw):
        x = {**d, **kw}
        o, hf = ssa.ssm_linattn_fwd(x["q"], x["k"], x["v"], x["log_decay"], h0=x["h0"])
        return (o.double() * d["dout"].double()).sum() + (hf.double() * d["dh_final"].double()).sum()

    gen = torch.Generator().manual_seed(19)
    args = (t["q"], t["k"], t["v"], t["log_decay"], K ** -0.5, t["dout"])
    m = ref.magnitude(ref.bwd, *args, h0=t["h0"], T=t["dh_final"])
    for x, n in (("q", "dq"), ("k", "dk"), ("v", "dv"), ("h0", "dh0")):
        step = torch.randn(t[x].shape, generator=gen)
        s = step.to(DEV)
        diff = (loss(**{x: d[x] + s}) - loss(**{x: d[x] - s})) / 2
        got = (g[n].double() * s.double()).sum()
        # each of the three sums is off by at most c times the same sum of absolute values; x + d and
        # x - d are rounded (2^-24 of at most |x| + |d|, in l by the same magnitudes)
        c = 2 * ref.term_error(L, K, V, False, extra=4)
        mag = float((m[n] * (step.double().abs() * 2 + t[x].double().abs())).sum())
        assert abs(float(diff - got)) <= c * mag, x


# ------------------------------------------------------------------ step and norm
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("B,H,G,K,V", [(1, 1, 1, 64, 64), (3, 4, 2, 128, 64), (2, 6, 1, 64, 128), (40, 16, 16, 128, 128)])
def test_step_and_its_norm(B, H, G, K, V, dtype):
    t = ref.inputs(B, 1, H, G, K, V, dtype, seed=B + H)
    d = dev(t)
    gen = torch.Generator().manual_seed(2)
    w, bias = torch.randn(H * V, generator=gen), torch.randn(H * V, generator=gen)
    z = torch.randn(B, H, V, generator=gen).to(dtype)
    one = [d[n][:, 0].contiguous() for n in ("q", "k", "v")]
    args = (t["q"], t["k"], t["v"], t["log_decay"], 0.25)
    ro, rs = ref.fwd(*args, h0=t["h0"])
    mo, ms = ref.magnitude(ref.fwd, *args, h0=t["h0"])
    state = d["h0"].clone()
    o = ssa.ssm_linattn_step(state, *one, d["log_decay"], scale=0.25)
    c = ref.term_error(1, K, V, False)
    ref.close(o[:, None], ro, mo, c, "o")
    ref.close(state, rs, ms, c, "state")
    for kw, wt, bt, zt in ((dict(), None, None, None), (dict(norm_weight=w.to(DEV), z=z.to(DEV)), w, None, z),
                           (dict(norm_weight=w.to(DEV), norm_bias=bias.to(DEV)), w, bias, None)):
        state = d["h0"].clone()
        y = ssa.ssm_linattn_step(state, *one, d["log_decay"], scale=0.25, norm_eps=1e-5, **kw)
        ref.close(state, rs, ms, c, "state")
        x = ro.reshape(B, 1, H * V)
        ry, mean, rstd = ref.norm_fwd(x, H, wt, bt, None if zt is None else zt.reshape(B, 1, H * V))
        # o is off by at most c mo; the norm moves by rstd |w| |gate| times that, its mean and spread by the
        # largest of the head's values (1 + |xhat| terms of it), and by its own sums
        worst = mo.reshape(B, 1, H, V).amax(3, keepdim=True).expand(B, 1, H, V).reshape(B, 1, H * V)
        xhat = ((x.reshape(B, 1, H, V) - mean[:, None, :, None]) * rstd[:, None, :, None]).reshape(B, 1, H * V)
        r = rstd[:, None, :, None].expand(B, 1, H, V).reshape(B, 1, H * V)
        gate = 1.0 if zt is None else (zt.double() * ref.sigmoid(zt.double())).abs().reshape(B, 1, H * V)
        wa = 1.0 if wt is None else wt.double().abs()
        ba = 0.0 if bt is None else bt.double().abs()
        s = ref.sum_error(V) + 20 * 2.0 ** -23
        mag = gate * (wa * r * worst * (2 + xhat.abs()) * (c + s) + (wa * (1 + xhat.abs()) + ba) * s)
        ref.close(y.reshape(B, 1, H * V), ry, mag, 1.0, "norm", store=dtype)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_forward_with_norm_is_the_two_calls(dtype):
    B, L, H, G, K, V = 2, 150, 4, 2, 64, 128
    t = dev(ref.inputs(B, L, H, G, K, V, dtype, seed=23))
    w, z = torch.randn(H * V, device=DEV), torch.randn(B, L, H, V, device=DEV).to(dtype)
    lens = lens_arg([150, 40])
    o, hf = ssa.ssm_linattn_fwd(t["q"], t["k"], t["v"], t["log_decay"], seqlens=lens, h0=t["h0"])
    y, _, _ = ssa.ssm_group_norm_fwd(o.reshape(B * L, H * V), H, w, None, z.reshape(B * L, H * V), eps=1e-6)
    y2, hf2 = ssa.ssm_linattn_fwd(t["q"], t["k"], t["v"], t["log_decay"], seqlens=lens, h0=t["h0"], norm_eps=1e-6,
                                  norm_weight=w, z=z)
    assert torch.equal(y.reshape(B, L, H, V), y2) and torch.equal(hf, hf2)


# ------------------------------------------------------------------ the ways it is called
def test_the_same_call_twice_gives_the_same_bits():
    t = dev(ref.inputs(2, 1000, 6, 2, 128, 64, BF16, seed=29))
    runs = [(ssa.ssm_linattn_fwd(t["q"], t["k"], t["v"], t["log_decay"], h0=t["h0"]),
             ssa.ssm_linattn_bwd(t["q"], t["k"], t["v"], t["log_decay"], t["dout"], h0=t["h0"],
                                 dh_final=t["dh_final"])) for _ in range(2)]
    (f1, g1), (f2, g2) = runs
    assert all(torch.equal(a, b) for a, b in zip(f1, f2)) and all(torch.equal(g1[n], g2[n]) for n in g1)


def test_on_a_side_stream_while_the_default_stream_allocates():
    t = dev(ref.inputs(2, 1000, 6, 2, 128, 64, BF16, seed=31))
    args = (t["q"], t["k"], t["v"], t["log_decay"])
    f = ssa.ssm_linattn_fwd(*args, h0=t["h0"])
    g = ssa.ssm_linattn_bwd(*args, t["dout"], h0=t["h0"], dh_final=t["dh_final"])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    f2 = ssa.ssm_linattn_fwd(*args, h0=t["h0"], stream=side)
    junk = [torch.full((1 << 20,), float("nan"), device=DEV) for _ in range(8)]
    g2 = ssa.ssm_linattn_bwd(*args, t["dout"], h0=t["h0"], dh_final=t["dh_final"], stream=side)
    junk += [torch.full((1 << 22,), float("nan"), device=DEV) for _ in range(8)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(f, f2)) and all(torch.equal(g[n], g2[n]) for n in g)


def test_two_streams_at_once():
    cases = [dev(ref.inputs(1, 1500 + 100 * i, 4, 2, 64, 64, BF16, seed=37 + i)) for i in range(2)]
    run = lambda t, s: ssa.ssm_linattn_fwd(t["q"], t["k"], t["v"], t["log_decay"], h0=t["h0"], stream=s)  # noqa: E731
    want = [run(t, None) for t in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = [[] for _ in cases]
    for _ in range(4):
        for i, (t, s) in enumerate(zip(cases, streams)):
            got[i].append(run(t, s))
    torch.cuda.synchronize()
    for w, gs in zip(want, got):
        assert all(torch.equal(a, b) for g in gs for a, b in zip(w, g))


def test_a_training_layer_and_a_decode_step_captured_and_replayed():
    """Attention, its gated norm, both gradients and a decode step with norm in one captured graph
    (workspaces of their own), replayed with eager work between; every replay gives the eager bits."""
    B, L, H, G, K, V = 2, 300, 4, 2, 128, 64
    t = dev(ref.inputs(B, L, H, G, K, V, BF16, seed=41))
    w, z = torch.randn(H * V, device=DEV), torch.randn(B * L, H * V, device=DEV).to(BF16)
    dy = torch.randn(B * L, H * V, device=DEV).to(BF16)
    one = [t[n][:, 0].contiguous() for n in ("q", "k", "v")]
    state = t["h0"].clone()

    def layer():
        o, hf = ssa.ssm_linattn_fwd(t["q"], t["k"], t["v"], t["log_decay"], h0=t["h0"])
        x = o.reshape(B * L, H * V)
        y, mean, rstd = ssa.ssm_group_norm_fwd(x, H, w, None, z)
        n = ssa.ssm_group_norm_bwd(x, H, mean, rstd, dy, w, None, z)
        g = ssa.ssm_linattn_bwd(t["q"], t["k"], t["v"], t["log_decay"], n["dx"].reshape(B, L, H, V), h0=t["h0"],
                                dh_final=t["dh_final"])
        state.copy_(t["h0"])
        s = ssa.ssm_linattn_step(state, *one, t["log_decay"], norm_eps=1e-5, norm_weight=w, z=one[2])
        return [o, hf, y, mean, rstd, *n.values(), *g.values(), s, state]

    eager = [x.clone() for x in layer()]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            out = layer()
    torch.cuda.synchronize()
    for rep in range(3):
        for x in out:
            x.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(out, eager)):
            assert torch.equal(a, b), f"replay {rep}, output {i}"
        layer()
        torch.cuda.synchronize()


def test_nothing_is_written_outside_the_outputs():
    """Outputs inside larger allocations: the bytes around them stay."""
    B, L, H, G, K, V = 1, 77, 3, 3, 64, 64
    t = dev(ref.inputs(B, L, H, G, K, V, BF16, seed=43))

    def framed(shape, dtype):
        n = 1
        for s in shape:
            n *= s
        buf = torch.full((n + 2048,), 7.0, dtype=dtype, device=DEV)
        return buf, buf[1024:1024 + n].view(shape)

    bufs, views = zip(*(framed(s, d) for s, d in (((B, L, H, V), BF16), ((B, H, K, V), F32), ((B, L, G, K), BF16),
                                                  ((B, L, G, K), BF16), ((B, L, H, V), BF16), ((B, H, K, V), F32))))
    ssa.ssm_linattn_fwd(t["q"], t["k"], t["v"], t["log_decay"], o=views[0], h_final=views[1])
    ssa.ssm_linattn_bwd(t["q"], t["k"], t["v"], t["log_decay"], t["dout"],
                        out=dict(dq=views[2], dk=views[3], dv=views[4], dh0=views[5]))
    torch.cuda.synchronize()
    for buf in bufs:
        assert (buf[:1024] == 7).all() and (buf[-1024:] == 7).all()


def test_offsets_beyond_32_bits():
    """More than 2^31 elements in v and o: the last rows are what a call on them alone gives from the
    state that the rows before leave."""
    L, H, V, tail = 140001, 120, 128, 130
    gen = torch.Generator(device=DEV).manual_seed(3)
    q, k = (torch.randn((1, L, 1, 64), generator=gen, device=DEV).to(BF16) for _ in range(2))
    v = torch.randn((1, L, H, V), generator=gen, device=DEV, dtype=BF16)
    assert v.numel() > 2 ** 31
    a = -torch.exp(torch.linspace(-8, 0, H, device=DEV))
    o, hf = ssa.ssm_linattn_fwd(q, k, v, a)
    _, s = ssa.ssm_linattn_fwd(q[:, :L - tail], k[:, :L - tail], v[:, :L - tail], a)
    o2, hf2 = ssa.ssm_linattn_fwd(q[:, L - tail:].contiguous(), k[:, L - tail:].contiguous(),
                                  v[:, L - tail:].contiguous(), a, h0=s)
    # both round the same values to bf16: a step apart at most, and rarely
    d = (o[:, L - tail:].float() - o2.float()).abs()
    assert float((d / (o2.float().abs() + o2.float().square().mean().sqrt())).max()) < 2.0 ** -6
    assert float((d > 0).float().mean()) < 0.05
    assert float((hf - hf2).norm() / hf.norm()) < 1e-6


@pytest.mark.parametrize("L", [70, 500])
@pytest.mark.parametrize("name", ["q", "k", "v"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_row_that_is_not_finite_leaves_the_chunks_before_it_and_the_other_rows_alone(L, name, bad):
    B, H, t = 2, 3, L - 5
    gen = torch.Generator(device=DEV).manual_seed(4)
    x = dict(q=torch.randn((B, L, H, 64), generator=gen, device=DEV).to(BF16),
             k=torch.randn((B, L, H, 64), generator=gen, device=DEV).to(BF16),
             v=torch.randn((B, L, H, 64), generator=gen, device=DEV).to(BF16))
    a = torch.tensor([0.0, -0.05, -1.0], device=DEV)
    want, hw = ssa.ssm_linattn_fwd(**x, log_decay=a)
    x[name][1, t, 2] = bad
    got, hg = ssa.ssm_linattn_fwd(**x, log_decay=a)
    before = t // 64 * 64
    assert torch.equal(got[0], want[0]) and torch.equal(got[1, :, :2], want[1, :, :2])
    assert torch.equal(got[1, :before, 2], want[1, :before, 2])
    assert not torch.isfinite(got[1, t, 2]).all()
    assert torch.equal(hg[0], hw[0]) and torch.equal(hg[1, :2], hw[1, :2])
    if name == "q":
        assert torch.equal(hg, hw)
    else:
        assert not torch.isfinite(hg[1, 2]).all()
