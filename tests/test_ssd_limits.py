"""How many (batch, head)s ssm_ssd_fwd takes: the refusal on any machine, the largest call on the GPU."""
import ctypes

import pytest
import torch

import selective_scan_amd as ssa
from selective_scan_amd import ops

P = ctypes.c_void_p(0x10000)


@pytest.mark.parametrize("B,H,status", [
    (65, 65535, 1),    # above 2^22
    (128, 65535, 1),   # 2^23 - 128
    (129, 65535, 2),   # above 2^23
    (65535, 129, 2),
])
def test_batches_times_heads(B, H, status):
    """x is missing (1), which is found after the sizes (2): no call reaches a launch."""
    assert ops.lib().ssm_ssd_fwd(B, 1, H, 64, 64, 0, 1, None, P, P, P, P, None, None, None, P, None, None, 0,
                                 None) == status
    assert ops.lib().ssm_last_error().startswith(b"ssm_ssd_fwd: " + (b"x," if status == 1 else b"B * H"))


@pytest.mark.gpu
def test_the_largest_number_of_workgroups():
    """One token of 2^23 - 128 (batch, head)s: batches of it are what calls on them alone give."""
    B, L, H, N = 128, 1, 65535, 64
    gen = torch.Generator(device="cuda:0").manual_seed(1)
    r = lambda *s: torch.randn(s, generator=gen, device="cuda:0", dtype=torch.bfloat16)  # noqa: E731
    x, delta, Bm, Cm = r(B, L, H, 64), r(B, L, H).abs(), r(B, L, N), r(B, L, N)
    A = -torch.rand(H, generator=gen, device="cuda:0")
    y, _ = ssa.ssm_ssd_fwd(x, delta, A, Bm, Cm, want_final_state=False)
    for b in (0, 64, 127):
        x1, d1, b1, c1 = (t[b:b + 1].clone() for t in (x, delta, Bm, Cm))
        y1, _ = ssa.ssm_ssd_fwd(x1, d1, A, b1, c1, want_final_state=False)
        torch.cuda.synchronize()
        assert torch.equal(y[b:b + 1], y1) and bool(y1.any())
