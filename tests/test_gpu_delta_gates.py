"""Gradients of the gated delta rule on the GPU where decays forget everything
(log decays far below fp32's range and minus infinity) and where beta is next to
0, against the fp64 adjoint.  Tolerances are those of
tests/test_gpu_delta_grads.py."""
import pytest
import torch

from tests.gpu_helpers import DEV
from tests.test_gpu_delta import make
from tests.test_gpu_delta_grads import TYPES, check_backward

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("B,L,H,Hk,dk,dv", [(1, 200, 4, 4, 64, 48), (1, 1500, 1, 1, 64, 64), (2, 70, 2, 1, 128, 128)])
def test_decays_that_forget_everything(B, L, H, Hk, dk, dv, dtype):
    T, tol = TYPES[dtype]
    x, g, b, s0, do, ds = make(B, L, H, Hk, dk, dv, T, seed=L)
    gen = torch.Generator().manual_seed(9)
    strong = torch.tensor([-120.0, -1000.0, -1e6, -1e30, float("-inf")])[torch.randint(0, 5, (B, L, H), generator=gen)].to(DEV)
    g = torch.where(torch.rand(B, L, H, generator=gen).to(DEV) < 0.05, strong, g)
    check_backward(x, g, b, s0, do, ds, tol)
    g[:, 0] = float("-inf")
    got = check_backward(x, g, b, s0, do, ds, tol)
    assert not bool(got[5].any())


@pytest.mark.parametrize("dtype", TYPES)
def test_betas_next_to_nothing(dtype):
    """beta of 0 and of numbers on either side of those that count as 0: the gradient of beta is v's part in all."""
    T, tol = TYPES[dtype]
    x, g, b, s0, do, ds = make(1, 150, 3, 3, 64, 48, T, seed=6)
    gen = torch.Generator().manual_seed(10)
    b = torch.tensor([0.0, 1e-30, 1e-20, -1e-20, 2e-20, 1e-12, -1e-25, 1.0])[torch.randint(0, 8, (1, 150, 3), generator=gen)].to(DEV)
    check_backward(x, g, b, s0, do, ds, tol)
