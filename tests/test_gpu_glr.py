"""Gated linear recurrence on the GPU against its 64-bit definition: whole sequences, gradient
and single tokens over types, forms, lengths around and far beyond the kernels' tiles, odd
widths, padding, strided rows and extreme gates."""
import pytest
import torch

import glr_ref as ref
import selective_scan_amd as ssa
from gpu_util import DEV

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
FORMS = ["decay", "convex"]


def to(t, dev=DEV):
    return {n: None if v is None else v.to(dev) for n, v in t.items()}


def lens(s):
    return None if s is None else torch.tensor(s, dtype=torch.int32, device=DEV)


def fwd(d, form, seqlens=None, **kw):
    return ssa.ssm_glr_fwd(d["x"], d["r"], d["i"], d["A"], d["z"], form=form, seqlens=lens(seqlens), h0=d["h0"],
                           want_states=True, **kw)


def bwd(d, states, form, seqlens=None, **kw):
    return ssa.ssm_glr_bwd(d["x"], d["r"], states, d["dy"], d["i"], d["A"], d["z"], form=form, seqlens=lens(seqlens),
                           dh_final=d["dh_final"], **kw)


def check(t, form, seqlens=None, what=""):
    dt = t["x"].dtype
    g = ref.Glr(t, form, seqlens, t["dy"], t["dh_final"])
    d = to(t)
    y, h, states = fwd(d, form, seqlens)
    torch.cuda.synchronize()
    ref.close(y, g.y, g.ey, 1.0, what + " y", store=dt)
    ref.close(h, g.h_final, g.eh_final, 1.0, what + " h_final", store=F32)
    ref.close(states, g.states, g.estates, 1.0, what + " states", store=F32)
    out = bwd(d, states, form, seqlens)
    torch.cuda.synchronize()
    for n in ("dx", "dr", "di", "dA", "dz", "dh0"):
        if n not in g.out:
            assert out[n] is None, n
            continue
        ref.close(out[n], *g.out[n], 1.0, f"{what} {n}", store=F32 if n in ("dA", "dh0") else dt)
    return y, h, states, out


SHAPES = [(1, 1, 1), (2, 3, 5), (1, 15, 64), (1, 16, 130), (3, 17, 128), (1, 127, 66), (1, 128, 257), (2, 129, 48),
          (3, 300, 100), (1, 1000, 200), (2, 640, 256), (1, 2500, 33), (2, 4097, 6), (1, 9000, 4)]


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_forward_and_gradient(shape, form, dtype):
    gate = sum(shape) % 2 == 0
    check(ref.glr_inputs(*shape, dtype, form, seed=sum(shape), gate=gate, h0=shape[2] % 2 == 0), form, what=str(shape))


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("gate", [True, False])
@pytest.mark.parametrize("h0", [True, False])
def test_every_combination_with_padding(form, gate, h0):
    for (B, L, D), s in (((4, 700, 40), [700, 0, 1, 333]), ((3, 129, 31), [128, 129, 127]), ((2, 20, 130), [-5, 99])):
        check(ref.glr_inputs(B, L, D, BF16, form, seed=L, gate=gate, h0=h0), form, s, what=f"{B}x{L}x{D}")


@pytest.mark.parametrize("form", FORMS)
def test_memories_of_one_token_and_of_the_whole_sequence(form):
    t = ref.glr_inputs(2, 3000, 32, F32, form, seed=5, fast=60.0, slow=1e-6)
    t["r"] = t["r"] * 4
    check(t, form)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("form", FORMS)
def test_gates_that_are_shut_or_open(form, dtype):
    """Gates from -infinity to infinity: values finite, closed gates hold the state exactly."""
    t = ref.glr_inputs(1, 400, 32, dtype, form, seed=6)
    vals = torch.tensor([-float("inf"), -300.0, -90.0, -40.0, 40.0, 90.0, 300.0, float("inf")]).to(dtype)
    t["r"][0, 100:200] = vals[torch.randint(8, (100, 32), generator=torch.Generator().manual_seed(1))]
    t["r"][0, 200:300] = -float("inf")
    if form == "decay":
        t["i"][0, 150:250] = vals[torch.randint(8, (100, 32), generator=torch.Generator().manual_seed(2))]
    y, h, states, out = check_finite(t, form)
    g = ref.Glr(t, form, None, t["dy"], t["dh_final"])
    ref.close(y, g.y, g.ey, 1.0, "y", store=dtype)
    for n in ("dx", "dz", "dh0"):
        ref.close(out[n], *g.out[n], 1.0, n, store=F32 if n == "dh0" else dtype)
    assert (out["dr"][0, 200:300] == 0).all() and (out["dx"][0, 200:300] == 0).all()


def check_finite(t, form):
    d = to(t)
    y, h, states = fwd(d, form)
    out = bwd(d, states, form)
    torch.cuda.synchronize()
    for v in (y, h, states, *out.values()):
        assert v is None or torch.isfinite(v).all()
    return y, h, states, out


def test_a_channel_without_decay():
    """A = 0: a = 1 and u = 0, the state stays; the gradient keeps to finite values."""
    t = ref.glr_inputs(1, 300, 8, F32, "decay", seed=7)
    t["A"][3] = 0.0
    y, h, states, out = check_finite(t, "decay")
    assert torch.equal(h[0, 3].cpu(), t["h0"][0, 3]) and (out["dx"][0, :, 3] == 0).all()


@pytest.mark.parametrize("form", FORMS)
def test_values_that_are_not_finite_keep_to_their_channel_sequence_and_later_steps(form):
    t = ref.glr_inputs(2, 500, 70, BF16, form, seed=8)
    a = to(t)
    clean = fwd(a, form)
    t["x"][0, 260, 5] = float("nan")
    t["r"][1, 499, 6] = float("nan")
    y, h, states = fwd(to(t), form)
    torch.cuda.synchronize()
    bad = torch.zeros_like(y, dtype=torch.bool)
    bad[0, 260:, 5] = True
    bad[1, 499, 6] = True
    assert torch.isnan(y[bad]).all() and torch.equal(y[~bad], clean[0][~bad])
    assert torch.isnan(h[0, 5]) and torch.isnan(h[1, 6]) and int(torch.isnan(h).sum()) == 2


@pytest.mark.parametrize("form", FORMS)
def test_padding_is_not_read(form):
    t = ref.glr_inputs(3, 300, 34, BF16, form, seed=9)
    s = [300, 131, 0]
    d = to(t)
    y, h, states = fwd(d, form, s)
    want = bwd(d, states, form, s)
    for b, n in enumerate(s):
        for k in ("x", "r", "i", "z", "dy"):
            if t[k] is not None:
                t[k][b, n:] = float("nan")
    d = to(t)
    y2, h2, states2 = fwd(d, form, s)
    got = bwd(d, states2, form, s)
    torch.cuda.synchronize()
    assert torch.equal(y, y2) and torch.equal(h, h2) and torch.equal(states, states2)
    for b, n in enumerate(s):
        assert (y2[b, n:] == 0).all()
    for k, v in want.items():
        if v is not None:
            assert torch.equal(v, got[k]), k
            if v.dim() == 3:
                assert all((v[b, n:] == 0).all() for b, n in enumerate(s))
    assert torch.equal(h2[2].cpu(), t["h0"][2]) and torch.equal(got["dh0"][2].cpu(), t["dh_final"][2])


def test_an_empty_sequence():
    t = ref.glr_inputs(2, 0, 6, BF16, "decay", seed=1)
    d = to(t)
    y, h, states = fwd(d, "decay")
    out = bwd(d, states, "decay")
    torch.cuda.synchronize()
    assert y.shape == (2, 0, 6) and torch.equal(h, d["h0"]) and states.shape == (2, 0, 6)
    assert torch.equal(out["dh0"], d["dh_final"]) and (out["dA"] == 0).all()


@pytest.mark.parametrize("form,gate", [("decay", True), ("convex", False)])
def test_tensors_that_outgrow_the_caches(form, gate):
    """More than 256 MiB in a call; a few channels of every kind of lane against 64 bits."""
    B, L, D = 2, 16500, 1502
    t = ref.glr_inputs(B, L, D, BF16, form, seed=14, gate=gate)
    s = [L, L - 777]
    d = to(t)
    y, h, states = fwd(d, form, s)
    out = bwd(d, states, form, s)
    torch.cuda.synchronize()
    pick = torch.tensor([0, 1, 62, 63, 64, 700, 1471, 1472, 1500, 1501])
    few = {n: None if v is None else v[..., pick].contiguous() for n, v in t.items()}
    g = ref.Glr(few, form, s, few["dy"], few["dh_final"])
    ref.close(y[..., pick.to(DEV)], g.y, g.ey, 1.0, "y", store=BF16)
    ref.close(h[..., pick.to(DEV)], g.h_final, g.eh_final, 1.0, "h_final", store=F32)
    for n, (v, e) in g.out.items():
        ref.close(out[n][..., pick.to(DEV)], v, e, 1.0, n, store=F32 if n in ("dA", "dh0") else BF16)


@pytest.mark.parametrize("D", [24, 27])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_slices_of_one_projection(D, dtype):
    t = ref.glr_inputs(2, 400, D, dtype, "decay", seed=10)
    d = to(t)
    wide = torch.cat([d["x"], d["r"], d["i"], d["z"]], 2)
    s = dict(d, **{n: wide[..., k * D:(k + 1) * D] for k, n in enumerate(("x", "r", "i", "z"))})
    want, got = fwd(d, "decay"), fwd(s, "decay")
    gw, gg = bwd(d, want[2], "decay"), bwd(s, got[2], "decay")
    torch.cuda.synchronize()
    for a, b in list(zip(want, got)) + [(gw[n], gg[n]) for n in gw]:
        assert torch.equal(a, b)
    state = d["h0"].clone()
    one = [wide[:, 7, k * D:(k + 1) * D] for k in range(4)]
    y1 = ssa.ssm_glr_step(state, one[0], one[1], one[2], d["A"], one[3])
    state2 = d["h0"].clone()
    y2 = ssa.ssm_glr_step(state2, *(o.contiguous() for o in one[:3]), d["A"], one[3].contiguous())
    torch.cuda.synchronize()
    assert torch.equal(y1, y2) and torch.equal(state, state2)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("B,D,gate", [(1, 1, True), (3, 257, False), (64, 512, True), (5, 1001, True)])
def test_steps_continue_a_sequence(B, D, gate, form, dtype):
    L, n = 40, 6
    t = ref.glr_inputs(B, L + n, D, dtype, form, seed=B + D, gate=gate)
    g = ref.Glr(t, form)
    d = to(t)
    head = {k: (v[:, :L].contiguous() if k in ("x", "r", "i", "z", "dy") and v is not None else v) for k, v in d.items()}
    _, state, _ = fwd(head, form)
    for s in range(L, L + n):
        tok = [None if d[k] is None else d[k][:, s] for k in ("x", "r", "i", "z")]
        y = ssa.ssm_glr_step(state, tok[0], tok[1], tok[2], d["A"], tok[3], form=form)
        torch.cuda.synchronize()
        ref.close(y, g.y[:, s], g.ey[:, s], 1.0, f"step {s}", store=dtype)
    ref.close(state, g.h_final, g.eh_final, 1.0, "state", store=F32)


def test_a_step_on_tokens_of_a_long_sequence():
    """Rows 5 million elements apart."""
    B, L, D = 2, 5000, 1024
    g = torch.Generator(device=DEV).manual_seed(4)
    x, r = (torch.randn((B, L, D), generator=g, device=DEV, dtype=BF16) for _ in range(2))
    a, b = (torch.zeros((B, D), device=DEV) for _ in range(2))
    y = ssa.ssm_glr_step(a, x[:, 77], r[:, 4321], form="convex")
    y2 = ssa.ssm_glr_step(b, x[:, 77].contiguous(), r[:, 4321].contiguous(), form="convex")
    torch.cuda.synchronize()
    assert torch.equal(y, y2) and torch.equal(a, b)


def test_the_gradient_is_the_difference_of_the_loss():
    """Along random directions, in fp32: (l(v + e d) - l(v - e d)) / 2 e against <gradient, d>. The
    loss is a sum of n products that are off by 2^-20 of their size at most, and its third
    derivative along unit directions is below 10 n. Along A that is no bound: a relative step v
    of A_d goes into terms like sqrt(1 + v), whose difference quotient is off by v^2 / 8 of the
    slope, and c e^-c (1 + v), off by v^2 c^2 / 6 of it, where c e^-c c^2 / 6 is at most 0.6 of
    the largest c e^-c: v^2 of what the terms of dA_d sum to without their signs."""
    for form in FORMS:
        t = ref.glr_inputs(1, 260, 16, F32, form, seed=12)
        d = to(t)
        states = fwd(d, form)[2]
        g = bwd(d, states, form)

        def loss(v):
            y, h, _ = fwd(v, form)
            return float((y.double() * d["dy"].double()).sum() + (h.double() * d["dh_final"].double()).sum())

        for n in ("x", "r", "i", "A", "z", "h0"):
            if d[n] is None:
                continue
            u = torch.randn(d[n].shape, generator=torch.Generator().manual_seed(3)).to(DEV)
            u = u / u.norm()
            e = 2.0 ** -5
            if n == "A":
                e = float((d["A"].abs() / u.abs()).min()) / 4
            num = (loss(dict(d, **{n: d[n] + e * u})) - loss(dict(d, **{n: d[n] - e * u}))) / (2 * e)
            want = float((g["d" + n].double() * u.double()).sum())
            size = float((g["d" + n].double() * u.double()).norm())
            y = fwd(d, form)[0].double()
            noise = float((y.abs() * d["dy"].double().abs()).norm()) * 2.0 ** -20 / e
            cut = 10 * e * e * max(size, abs(want), 1.0)
            if n == "A":
                mag = ref.Glr(t, form, None, t["dy"], t["dh_final"]).magA.to(DEV)
                cut = float(((e * u / d["A"]).double() ** 2 * u.double().abs() * mag).sum())
            assert abs(num - want) <= noise + cut, (form, n, num, want)


def test_results_repeat_bit_for_bit():
    t = ref.glr_inputs(3, 5000, 300, BF16, "decay", seed=13)
    d = to(t)
    first = fwd(d, "decay")
    g1 = bwd(d, first[2], "decay")
    for _ in range(3):
        again = fwd(d, "decay")
        g2 = bwd(d, again[2], "decay")
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(first, again))
        assert all(torch.equal(g1[n], g2[n]) for n in g1)


def test_two_streams_at_once_and_a_dirty_workspace():
    t = [ref.glr_inputs(2, 6000, 200 + 56 * k, BF16, "decay", seed=20 + k) for k in range(2)]
    d = [to(v) for v in t]
    want = [fwd(v, "decay") for v in d]
    gw = [bwd(v, w[2], "decay") for v, w in zip(d, want)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got, gg, keep = [None] * 2, [None] * 2, []
    for rep in range(3):
        for k, s in enumerate(streams):
            B, L, D = d[k]["x"].shape
            ws = torch.full((ssa.ssm_glr_workspace_size(B, L, D) + 16,), 255 if rep else 0, dtype=torch.uint8, device=DEV)
            wb = torch.full((ssa.ssm_glr_bwd_workspace_size(B, L, D) + 16,), 255 if rep else 0, dtype=torch.uint8, device=DEV)
            keep += [ws, wb]
            s.wait_stream(torch.cuda.current_stream())
            got[k] = fwd(d[k], "decay", stream=s, workspace=ws)
            gg[k] = bwd(d[k], got[k][2], "decay", stream=s, workspace=wb)
        torch.cuda.synchronize()
        for k in range(2):
            assert all(torch.equal(a, b) for a, b in zip(want[k], got[k]))
            assert all(torch.equal(gw[k][n], gg[k][n]) for n in gw[k])


def test_captured_and_replayed():
    t = ref.glr_inputs(2, 3000, 130, BF16, "decay", seed=30)
    d = to(t)
    state = d["h0"].clone()
    tok = {n: d[n][:, 0].contiguous() for n in ("x", "r", "i", "z")}

    def work():
        y, h, states = fwd(d, "decay")
        g = bwd(d, states, "decay")
        return [y, h, states, *g.values(), ssa.ssm_glr_step(state, tok["x"], tok["r"], tok["i"], d["A"], tok["z"]), state]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        work()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        outs = work()
    for rep in range(3):
        fresh = ref.glr_inputs(2, 3000, 130, BF16, "decay", seed=31 + rep)
        for n, v in fresh.items():
            d[n].copy_(v)
        for n in tok:
            tok[n].copy_(fresh[n][:, 0])
        state.copy_(fresh["h0"])
        want = [v.clone() for v in work()]
        state.copy_(fresh["h0"])
        for o in outs[:-1]:
            o.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(want, outs):
            assert torch.equal(a, b), rep
        _ = (want[0].float() * 2).sum().item()


def test_outputs_of_the_caller_and_what_is_not_wanted():
    t = ref.glr_inputs(2, 300, 36, BF16, "decay", seed=40)
    d = to(t)
    y, h, states = fwd(d, "decay")
    buf = torch.full_like(y, 7.0)
    y2, h2, s2 = ssa.ssm_glr_fwd(d["x"], d["r"], d["i"], d["A"], d["z"], h0=d["h0"], y=buf, want_final_state=False)
    assert y2 is buf and h2 is None and s2 is None
    g = bwd(d, states, "decay")
    out = {"dx": torch.full_like(y, 7.0)}
    g2 = bwd(d, states, "decay", out=out, want_dh0=False)
    torch.cuda.synchronize()
    assert torch.equal(y, buf) and g2["dx"] is out["dx"] and torch.equal(g["dx"], g2["dx"]) and g2["dh0"] is None


@pytest.mark.parametrize("D", [36, 65, 130])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_nothing_is_written_around_the_outputs_and_nothing_read_between_the_rows(D, dtype):
    """Every output lies between guards; every input is a slice of rows whose rest is NaN, at an
    odd and at an even place."""
    B, L = 2, 333
    t = ref.glr_inputs(B, L, D, dtype, "decay", seed=50)
    d = to(t)
    s = [L, 200]
    y, h, states = fwd(d, "decay", s)
    want = dict(y=y, h_final=h, states=states, **bwd(d, states, "decay", s))
    for at in (3, 8):
        wide = {n: torch.full((B, L, D + 16), float("nan"), dtype=dtype, device=DEV) for n in ("x", "r", "i", "z")}
        e = dict(d)
        for n, v in wide.items():
            v[..., at:at + D] = d[n]
            e[n] = v[..., at:at + D]
        bufs = {n: torch.full((v.numel() + 128,), 7.0, dtype=v.dtype, device=DEV) for n, v in want.items()}
        out = {n: b[64:64 + want[n].numel()].view(want[n].shape) for n, b in bufs.items()}
        fwd(e, "decay", s, y=out["y"], h_final=out["h_final"], states=out["states"])
        bwd(e, out["states"], "decay", s, out={n: out[n] for n in ("dx", "dr", "di", "dA", "dz", "dh0")})
        torch.cuda.synchronize()
        for n, b in bufs.items():
            assert (b[:64] == 7).all() and (b[64 + want[n].numel():] == 7).all(), n
            # strided rows that are no pairs take the single-channel kernels, whose sums run in
            # another order: equal to a rounding of the fp32 values behind them, in storage to a step
            a, c = out[n].double(), want[n].double()
            tol = torch.finfo(want[n].dtype).eps * c.abs() + 2.0 ** -17 * c.abs().mean()
            assert ((a - c).abs() <= tol).all(), n


@pytest.mark.parametrize("form", FORMS)
def test_a_sequence_in_two_parts(form):
    t = ref.glr_inputs(2, 900, 50, F32, form, seed=51)
    g = ref.Glr(t, form)
    d = to(t)
    for cut in (1, 128, 517, 899):
        a, b = ({n: v[:, sl].contiguous() if n in ("x", "r", "i", "z", "dy") and v is not None else v for n, v in d.items()}
                for sl in (slice(0, cut), slice(cut, None)))
        y1, h1, _ = fwd(a, form)
        y2, h2, _ = fwd(dict(b, h0=h1), form)
        torch.cuda.synchronize()
        ref.close(torch.cat([y1, y2], 1), g.y, 2 * g.ey, 1.0, f"y cut at {cut}", store=F32)
        ref.close(h2, g.h_final, 2 * g.eh_final, 1.0, f"h_final cut at {cut}", store=F32)
