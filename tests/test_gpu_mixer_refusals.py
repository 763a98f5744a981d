"""Outputs of the delta-rule mixer's operators that would be written over what
the call still reads are refused; neighbours in one allocation are not."""
import pytest
import torch

from nonlinear_rnn_solve_pararnn_amd import api
from tests.gpu_helpers import DEV
from tests.test_gpu_delta import make

pytestmark = pytest.mark.gpu


def test_outputs_over_inputs():
    x, g, b, s0, do, ds = make(2, 40, 2, 2, 16, 16, torch.float32, seed=50)
    q, k, v = x
    for bad in (q, k, v):
        with pytest.raises(api.PararnnError):
            api.delta_forward(q, k, v, g, b, s0, out=bad)
        with pytest.raises(api.PararnnError):
            api.headnorm_forward(q, k, out_q=bad if bad is not v else k)
    q1, k1, v1, g1, b1 = (t[:, 0].contiguous() for t in (q, k, v, g, b))
    with pytest.raises(api.PararnnError):
        api.delta_step(q1, k1, v1, g1, b1, s0, out=v1)
    rest = torch.empty(s0.numel() + 2 * 40 * 2 * 16, device=DEV)
    with pytest.raises(api.PararnnError):  # the output over the end of the state
        api.delta_forward(q, k, v, g, b, rest[:s0.numel()].view(s0.shape), out=rest[-v.numel() - 1:-1].view(v.shape))
    same = torch.empty(2, 40, 2, 16, device=DEV)
    with pytest.raises(api.PararnnError):
        api.headnorm_forward(q, k, out_q=same, out_k=same)


def test_neighbours_in_one_allocation():
    x, g, b, s0, do, ds = make(2, 40, 2, 2, 16, 16, torch.float32, seed=51)
    want = api.delta_forward(*x, g, b, s0)
    n = x[0].numel()
    buf = torch.empty(4 * n + 2 * s0.numel(), device=DEV)
    parts = [buf[i * n:(i + 1) * n].view(x[0].shape) for i in range(4)]
    for p, t in zip(parts, x):
        p.copy_(t)
    states = [buf[4 * n + i * s0.numel():4 * n + (i + 1) * s0.numel()].view(s0.shape) for i in range(2)]
    states[0].copy_(s0)
    o, s = api.delta_forward(*parts[:3], g, b, states[0], out=parts[3], out_state=states[1])
    assert o is parts[3] and s is states[1]
    assert torch.equal(o, want[0]) and torch.equal(s, want[1])
    a, c = api.headnorm_forward(parts[0], parts[1], out_q=parts[2], out_k=parts[3]), api.headnorm_forward(x[0], x[1])
    assert torch.equal(a[0], c[0]) and torch.equal(a[1], c[1])
