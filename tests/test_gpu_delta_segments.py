"""The gated delta rule of wide heads in segments, on the GPU, at lengths from
which they are taken there (tests/test_delta_segments.py), against the fp64
formulas, with states and shared keys.  Tolerances are those of
tests/test_gpu_delta.py and tests/test_gpu_delta_grads.py."""
import pytest
import torch

from nonlinear_rnn_solve_pararnn_amd import api
from tests.test_delta_segments import BF16, F32, in_segments
from tests.test_gpu_delta import BF16_TOL, F32_TOL, check_forward, make
from tests.test_gpu_delta_grads import check_backward

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("L,H,dk,dv", [(2100, 1, 256, 130), (2099, 2, 200, 24), (2051, 1, 129, 256)])
def test_wide_heads_forward(L, H, dk, dv):
    for T, code, tol in ((torch.float32, F32, F32_TOL), (torch.bfloat16, BF16, BF16_TOL)):
        assert in_segments(0, code, L, H, dk, dv)
        x, g, b, s0, _, _ = make(1, L, H, 1, dk, dv, T, seed=L)
        check_forward(x, g, b, s0, tol)


@pytest.mark.parametrize("dtype,L,H,dk,dv", [("f32", 2100, 1, 256, 130), ("f32", 2099, 2, 200, 24), ("bf16", 3700, 1, 256, 130), ("bf16", 3699, 2, 200, 24)])
def test_wide_heads_backward(dtype, L, H, dk, dv):
    T, code, tol = (torch.float32, F32, 1.6e-5) if dtype == "f32" else (torch.bfloat16, BF16, 4e-3)
    assert in_segments(1, code, L, H, dk, dv)
    check_backward(*make(1, L, H, 1, dk, dv, T, seed=L), tol)


@pytest.mark.parametrize("dtype", ("f32", "bf16"))
def test_values_that_are_not_finite_in_wide_segments(dtype):
    T = torch.float32 if dtype == "f32" else torch.bfloat16
    x, g, b, s0, _, _ = make(1, 2100, 1, 1, 256, 40, T, seed=3)
    clean, sclean = api.delta_forward(*x, g, b, s0)
    y = [z.clone() for z in x]
    y[2][0, 900, 0, 7] = float("inf")
    o, s = api.delta_forward(*y, g, b, s0)
    rest = [c for c in range(40) if c != 7]
    assert torch.equal(o[:, :900], clean[:, :900]) and torch.equal(o[..., rest], clean[..., rest]) and torch.equal(s[..., rest], sclean[..., rest])
    assert not bool(torch.isfinite(o[0, 900:, 0, 7]).any()) and not bool(torch.isfinite(s[0, 0, :, 7]).any())
