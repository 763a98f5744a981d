"""The gated delta rule's backward pass on the GPU with more spans than
workgroups, so that a workgroup goes on from span to span and from one pair of
batch row and head to the next; and its gradients as slopes, along themselves.

Tolerances of the parity tests are those of tests/test_gpu_delta_grads.py."""
import pytest
import torch

from nonlinear_rnn_solve_pararnn_amd import api
from tests.test_gpu_delta import make
from tests.test_gpu_delta_grads import TYPES, check_backward

pytestmark = pytest.mark.gpu


# spans of 64 positions (fp32 32): 432 on 256 workgroups (bf16, heads above 64), 768 and 1344 on 512 or 768 (up to 64),
# with lengths that end inside a span, shared heads, and gates whose strides are not those of dense tensors
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("B,L,H,Hk,dk,dv", [(6, 330, 12, 6, 128, 96), (16, 200, 12, 12, 64, 64), (20, 129, 15, 5, 24, 40), (300, 65, 2, 2, 72, 8)])
def test_several_spans_a_workgroup(B, L, H, Hk, dk, dv, dtype):
    T, tol = TYPES[dtype]
    x, g, b, s0, do, ds = make(B, L, H, Hk, dk, dv, T, seed=B + L)
    gates = torch.stack([g, b], -1)
    first = check_backward(x, gates[..., 0], gates[..., 1], s0, do, ds, tol)
    for _ in range(3):
        for a, c in zip(api.delta_backward(*x, g, b, do, s0, ds), first):
            assert torch.equal(a, c)


@pytest.mark.parametrize("dtype", TYPES)
def test_a_gradient_is_the_slope_along_itself(dtype):
    """Steps of h (a root of squares an element) along each operand's gradient; with bf16 tensors along those of the
    fp32 operands, whose steps are not rounded.  The difference of the losses is the gradient's product with the step
    up to terms of the third order, a few times h^2 of it in keys of 32 elements of 1 / sqrt(32) (5e-3 in all), and
    what rounding leaves of the outputs: half a step of each, independent, four times their root of squares."""
    T, _ = TYPES[dtype]
    x, g, b, s0, do, ds = make(1, 70, 2, 1, 32, 40, T, seed=7)
    args = [*x, g, b, s0]
    grads = api.delta_backward(*x, g, b, do, s0, ds)
    o, s = api.delta_forward(*args[:5], s0)
    half = torch.finfo(T).eps / 2
    noise = 4 * (2.0 ** 0.5) * (half * float((o.double() * do.double()).norm()) + 2.0 ** -21 * float((s.double() * ds.double()).norm()))
    if T == torch.float32:
        noise *= 8  # sums of some tens of roundings

    def loss(a):
        o, s = api.delta_forward(*a[:5], a[5])
        return float((o.double() * do.double()).sum() + (s.double() * ds.double()).sum())

    h = 2e-3 if T == torch.float32 else 2e-2
    for i in range(6) if T == torch.float32 else range(3, 6):
        n = grads[i].numel()
        step = (h * n ** 0.5 / grads[i].double().norm()).float() * grads[i].float()
        up, down = list(args), list(args)
        up[i], down[i] = args[i] + step, args[i] - step
        want = float((grads[i].double() * step.double()).sum())
        slope = (loss(up) - loss(down)) / 2
        assert abs(slope - want) <= 5e-3 * want + noise, (i, slope, want, noise)
        assert noise < 0.05 * want, (i, noise, want)
