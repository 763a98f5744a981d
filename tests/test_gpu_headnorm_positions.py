"""Head norms on the GPU with positions of any strides: a row's for all rows, a
column of a batch's, every other one."""
import pytest
import torch

from nonlinear_rnn_solve_pararnn_amd import api, sequence
from tests.gpu_helpers import DEV
from tests.test_gpu_headnorm import make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bits", [torch.int32, torch.int64])
def test_positions_of_any_strides(bits):
    x, dy, w, tab, pos = make(3, 7, 4, 2, 32, 16, torch.float32, seed=8, P=60)
    row = torch.arange(7, device=DEV).to(bits)
    wide = torch.randint(0, 60, (7, 6), device=DEV).to(bits)
    for p in (row.expand(3, 7), wide[:, ::2].t(), row.flip(0)[None].expand(3, 7)):
        assert not p.is_contiguous()
        got, want = (api.headnorm_forward(*x, *w, tab, t) for t in (p, p.clone(memory_format=torch.contiguous_format)))
        back = [api.headnorm_backward(*x, got[2], got[3], *dy, *w, tab, t) for t in (p, p.clone(memory_format=torch.contiguous_format))]
        for a, c in zip((*got, *back[0]), (*want, *back[1])):
            assert torch.equal(a, c)
    one = api.headnorm_forward(x[0][:, 2], x[1][:, 2], *w, tab, wide[:3, 1])
    same = api.headnorm_forward(x[0][:, 2], x[1][:, 2], *w, tab, wide[:3, 1].contiguous())
    assert torch.equal(one[0], same[0]) and torch.equal(one[1], same[1])


def test_modules_take_a_column_of_positions():
    torch.manual_seed(0)
    mix = sequence.LinearAttention(32, 2, 16, norm="rms", rotary=16, max_positions=64, device=DEV)
    x = torch.randn(2, 5, 32, device=DEV)
    pos = torch.arange(5, device=DEV).expand(2, 5)
    y, s = mix(x, None, pos)
    assert torch.equal(y, mix(x)[0])
    y.square().sum().backward()
    again = mix(x[:, :4], None, pos[:, :4])[1].detach()
    y4, s4 = mix.step(x[:, 4], again, pos[:, 4])
    # states and outputs of size 1, sums of some tens of products in fp32: 1e-5 is 80 roundings of 2^-23
    assert torch.allclose(y4, y[:, 4], rtol=0, atol=1e-5) and torch.allclose(s4, s, rtol=0, atol=1e-5)
