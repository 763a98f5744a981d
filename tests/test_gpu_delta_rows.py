"""The gated delta rule on the GPU with rows that are one row in memory, and with
positions of a padded batch that hold anything.

Tolerances are those of the operators' own tests (tests/test_gpu_delta.py,
tests/test_gpu_delta_grads.py)."""
import pytest
import torch

from nonlinear_rnn_solve_pararnn_amd import api, sequence
from tests import mixer_ref as ref
from tests.gpu_helpers import DEV
from tests.lm_ref import f64, rel
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


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("L,H,Hk,dk,dv", [(100, 2, 2, 64, 64), (75, 2, 1, 24, 40), (1500, 1, 1, 128, 64)])
def test_gradients_of_padded_rows_whatever_stands_there(L, H, Hk, dk, dv, dtype):
    """beta = 0 and log_decay = 0 leave the state as it is: the other positions' gradients are those of zeros there."""
    fwd, back = TOL[dtype]
    x, g, b, s0, do, ds = make(2, L, H, Hk, dk, dv, TYPES[dtype], seed=L)
    off = torch.zeros(2, L, dtype=torch.bool, device=DEV)
    off[1, L // 3:L // 3 + 7] = off[1, L - 20:] = off[0, 5] = True
    g[off], b[off], do[off] = 0.0, 0.0, 0.0
    want = check_backward(x, g, b, s0, do, ds, back)
    for value in (torch.finfo(TYPES[dtype]).min, 1e30, -1e18):
        y = [t.clone() for t in x]
        y[2][off] = value
        o, s = api.delta_forward(*y, g, b, s0)
        got = api.delta_backward(*y, g, b, do, s0, ds, want_state=True)
        clean = api.delta_forward(*x, g, b, s0)
        assert torch.equal(s, clean[1]) and torch.equal(o[~off], clean[0][~off])
        for i in range(5):  # beta's own gradient is v's product there
            assert torch.equal(got[i][~off], want[i][~off]), (value, i)
            assert i == 4 or torch.equal(got[i][off], want[i][off]), (value, i)
        assert torch.equal(got[5], want[5])
        if abs(value) < 1e38:  # or the gradient itself is past fp32
            want_gb = ref.delta_grads(*f64(*y), *f64(g, b, do, s0, ds))[4]
            assert rel(got[4][off], want_gb[off.cpu()]) <= 1.6e-5
