"""Rounding of the gated delta rule's bf16 outputs on the GPU: once, from fp32.

Every case has unit keys and queries with a single one in them, no decay, and
sums of one term, so the fp32 value of each element is a number of the inputs
without any rounding, and the output is that number's nearest bf16: no
tolerance.  The numbers stand just above the middle between two bf16, where an
operand of 16 bits falls on it and rounds to the lower one, and anywhere."""
import pytest
import torch

from nonlinear_rnn_solve_pararnn_amd import api
from tests.gpu_helpers import DEV

pytestmark = pytest.mark.gpu


def numbers(n, gen):
    """Numbers in (1, 2): half of them 2^-20 above a middle, half anywhere."""
    middle = 1.0 + torch.randint(0, 128, (n,), generator=gen) / 128.0 + 2.0 ** -8 + 2.0 ** -20
    return torch.where(torch.rand(n, generator=gen) < 0.5, middle, 1.0 + torch.rand(n, generator=gen))


def one_hot(at, d):
    return torch.nn.functional.one_hot(at, d).to(torch.bfloat16).to(DEV)


@pytest.mark.parametrize("B,L,H,dk,dv", [(1, 70, 2, 48, 72), (1, 33, 3, 128, 128), (2, 40, 1, 200, 24), (1, 1500, 1, 32, 40)])
def test_outputs_read_the_state_in_32_bits(B, L, H, dk, dv):
    gen = torch.Generator().manual_seed(L)
    s0 = numbers(B * H * dk * dv, gen).view(B, H, dk, dv).to(DEV)
    at = torch.randint(0, dk, (B, L, H), generator=gen)
    q, k = one_hot(at, dk), one_hot(torch.randint(0, dk, (B, L, H), generator=gen), dk)
    zeros = torch.zeros(B, L, H, device=DEV)
    o, s = api.delta_forward(q, k, torch.ones(B, L, H, dv, dtype=torch.bfloat16, device=DEV), zeros, zeros, s0, scale=1.0)
    want = s0.gather(2, at.to(DEV).permute(0, 2, 1)[..., None].expand(B, H, L, dv)).transpose(1, 2)
    assert torch.equal(s, s0) and torch.equal(o, want.to(torch.bfloat16))


@pytest.mark.parametrize("L,dk,dv", [(32, 64, 8), (60, 64, 72), (128, 128, 128), (200, 200, 33)])
def test_outputs_take_writes_and_weights_in_32_bits(L, dk, dv):
    """Position t writes b_t at key t; outputs ask for the keys of their own chunk and of earlier ones."""
    gen = torch.Generator().manual_seed(L)
    b = numbers(L * 2, gen).view(1, L, 2).to(DEV)
    t = torch.arange(L)
    ask = (torch.rand(L, generator=gen) * (t + 1)).long()
    ask[::2] = t[::2] // 32 * 32 + (torch.rand(L, generator=gen)[::2] * (t[::2] % 32 + 1)).long()
    q, k = (one_hot(i[None, :, None].expand(1, L, 2), dk) for i in (ask, t))
    sign = torch.where(torch.rand(1, L, 2, dv, generator=gen) < 0.5, -1.0, 1.0).to(torch.bfloat16).to(DEV)
    g = torch.zeros(1, L, 2, device=DEV)
    o, _ = api.delta_forward(q, k, sign, g, b, scale=1.0)
    assert torch.equal(o, (b[..., None] * sign.float())[:, ask].to(torch.bfloat16))
    for scale in (1.0 + 2.0 ** -8 + 2.0 ** -20, 1.0 + 5 * 2.0 ** -8 + 2.0 ** -20):
        o, _ = api.delta_forward(q, k, sign, g, torch.ones_like(b), scale=scale)
        assert torch.equal(o, (scale * sign.float())[:, ask].to(torch.bfloat16))


@pytest.mark.parametrize("L,dk,dv", [(32, 64, 8), (60, 64, 72), (128, 128, 128), (200, 200, 33)])
def test_gradients_take_pairs_in_32_bits(L, dk, dv):
    """One output has a gradient, of one element: its query's gradient at key t is what position t wrote there."""
    gen = torch.Generator().manual_seed(L + 1)
    b = numbers(L * 2, gen).view(1, L, 2).to(DEV)
    t = torch.arange(L)
    q = k = one_hot(t[None, :, None].expand(1, L, 2), dk)
    v = torch.ones(1, L, 2, dv, dtype=torch.bfloat16, device=DEV)
    do = torch.zeros(1, L, 2, dv, dtype=torch.bfloat16, device=DEV)
    do[:, L - 1, :, 3] = 1.0
    dq = api.delta_backward(q, k, v, torch.zeros(1, L, 2, device=DEV), b, do, scale=1.0)[0]
    want = torch.zeros_like(dq)
    want[0, L - 1, :, :L] = b[0].t().to(torch.bfloat16)
    assert torch.equal(dq, want)
