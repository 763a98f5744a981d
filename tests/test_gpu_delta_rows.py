"""The gated delta rule on the GPU with rows that are one row in memory.

Tolerances are those of the operators' own tests (tests/test_gpu_delta.py,
tests/test_gpu_delta_grads.py)."""
import pytest
import torch

from nonlinear_rnn_solve_pararnn_amd import sequence
from tests import mixer_ref as ref
from tests.gpu_helpers import DEV
from tests.lm_ref import rel
from tests.test_gpu_delta import BF16_TOL, F32_TOL, check_forward, make
from tests.test_gpu_delta_grads import check_backward

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
TOL = {"f32": (F32_TOL, 1.6e-5), "bf16": (BF16_TOL, 4e-3)}


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("L,H,Hk,dk,dv", [(1, 2, 2, 64, 64), (33, 4, 2, 32, 48), (70, 2, 2, 128, 128), (70, 2, 1, 24, 40), (70, 1, 1, 17, 33), (1500, 2, 2, 64, 64)])
def test_operands_expanded_over_the_positions(L, H, Hk, dk, dv, dtype):
    """Each of q, k, v and grad_o one row for all positions, alone and together."""
    fwd, back = TOL[dtype]
    x, g, b, s0, do, ds = make(2, L, H, Hk, dk, dv, TYPES[dtype], seed=L + dk)
    one = lambda t: t[:, :1].expand(t.shape)  # noqa: E731
    for names in ("qo", "kv", "qkvo") if L > 100 else ("q", "k", "v", "o", "qo", "kv", "ko", "qkvo"):
        y = [one(t) if n in names else t for n, t in zip("qkv", x)]
        y_do = one(do) if "o" in names else do
        check_forward(y, g, b, s0, fwd)
        check_backward(y, g, b, s0, y_do, ds, back)


def test_a_mean_over_the_positions_of_one_query():
    """The loss whose gradient is one row for all positions, through autograd."""
    x, g, b, s0, _, _ = make(2, 70, 2, 2, 64, 48, torch.float32, seed=3)
    leaves = [t.detach().requires_grad_(True) for t in (x[0][:, :1], x[1], x[2], g, b, s0)]
    o, _ = sequence.gated_delta(leaves[0].expand(2, 70, 2, 64), *leaves[1:])
    o.mean(1).square().sum().backward()
    plain = [t.detach().cpu().double().requires_grad_(True) for t in leaves]
    o, _ = ref.delta(plain[0].expand(2, 70, 2, 64), *plain[1:])
    o.mean(1).square().sum().backward()
    for a, c in zip(leaves, plain):
        assert rel(a.grad, c.grad) <= 4 * TOL["f32"][1]  # the gradient that comes in is off as well, and a sum over 70 positions
