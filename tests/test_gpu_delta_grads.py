"""GPU parity of the gated delta rule's gradients against the fp64 adjoint.

Tolerances, relative in the 2-norm.  fp32 results of fp32 tensors: sums of some
hundred products as in the forward pass, behind two recurrences instead of one:
256 * 2^-24 = 1.6e-5.  With bf16 tensors the gradients of the gates come from
factors of 16 bits, at most 2^-17 of each of two in a product: 1.6e-5 as well;
gradients of q, k and v are rounded once (2^-8 = 3.9e-3 of the value at the most)
from sums of such products: 4e-3.
The gradient of the state is fp32 in both."""
import pytest
import torch

from nonlinear_rnn_solve_pararnn_amd import api
from tests import mixer_ref as ref
from tests.gpu_helpers import DEV, say
from tests.lm_ref import f64, rel
from tests.test_gpu_delta import SHAPES, make

pytestmark = pytest.mark.gpu

F32_TOL, BF16_TOL = 1.6e-5, 4e-3
TYPES = {"f32": (torch.float32, F32_TOL), "bf16": (torch.bfloat16, BF16_TOL)}


def check_backward(x, g, b, s0, do, ds, tol, **kw):
    got = api.delta_backward(*x, g, b, do, s0, ds, want_state=True, **kw)
    want = ref.delta_grads(*f64(*x), *f64(g, b, do, s0, ds), scale=kw.get("scale"))
    errs = [rel(a, c) for a, c in zip(got, want)]
    say("backward", tuple(x[0].shape), tuple(x[2].shape[2:]), x[0].dtype, errs)
    assert [t.dtype for t in got] == [x[0].dtype] * 3 + [torch.float32] * 3
    assert max(errs[:3]) <= tol and max(errs[3:]) <= F32_TOL, errs
    return got


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("B,L,H,Hk,dk,dv", SHAPES)
def test_backward(B, L, H, Hk, dk, dv, dtype):
    T, tol = TYPES[dtype]
    check_backward(*make(B, L, H, Hk, dk, dv, T, seed=L * 7 + dk), tol)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("L,H,Hk,dk,dv", [(2051, 1, 1, 64, 128), (1500, 2, 1, 128, 40), (1600, 2, 2, 33, 31)])
def test_long_sequence_with_few_rows(L, H, Hk, dk, dv, dtype):
    T, tol = TYPES[dtype]
    check_backward(*make(1, L, H, Hk, dk, dv, T, seed=L), tol)


@pytest.mark.parametrize("dtype", TYPES)
def test_without_states_and_with_a_scale(dtype):
    T, tol = TYPES[dtype]
    x, g, b, _, do, _ = make(2, 150, 3, 3, 64, 64, T, seed=5, state=False)
    check_backward(x, g, b, None, do, None, tol, scale=0.3)
    assert api.delta_backward(*x, g, b, do)[5] is None


@pytest.mark.parametrize("dtype", TYPES)
def test_gates_at_their_ends(dtype):
    """beta of 0, 1 and 2; no decay and strong ones beside slow ones."""
    T, tol = TYPES[dtype]
    x, g, b, s0, do, ds = make(1, 200, 4, 4, 64, 48, T, seed=6)
    gen = torch.Generator().manual_seed(8)
    b = torch.tensor([0.0, 1.0, 2.0, 0.5])[torch.randint(0, 4, (1, 200, 4), generator=gen)].to(DEV)
    g = torch.tensor([0.0, -1e-6, -0.01, -0.5, -8.0, -60.0])[torch.randint(0, 6, (1, 200, 4), generator=gen)].to(DEV)
    g[:, :, 1:] = torch.where(torch.rand(1, 200, 3, generator=gen).to(DEV) < 0.9, torch.full_like(g[:, :, 1:], -1e-3), g[:, :, 1:])
    got = check_backward(x, g, b, s0, do, ds, tol)
    assert bool((got[2].float()[b == 0] == 0).all())  # v is not written there


@pytest.mark.parametrize("dtype", TYPES)
def test_a_gradient_is_the_slope(dtype):
    """The loss along a direction, from the forward kernel, against the gradients' product with it."""
    x, g, b, s0, do, ds = make(1, 70, 2, 1, 32, 40, torch.float32, seed=7)
    grads = api.delta_backward(*x, g, b, do, s0, ds)
    gen = torch.Generator().manual_seed(9)

    def loss(args):
        o, s = api.delta_forward(*args[:5], args[5])
        return float((o.double() * do.double()).sum() + (s.double() * ds.double()).sum())

    args = [*x, g, b, s0]
    for i in range(6):
        step = torch.randn(args[i].shape, generator=gen).to(DEV) * 0.02
        up, down = list(args), list(args)
        up[i], down[i] = args[i] + step, args[i] - step
        slope = (loss(up) - loss(down)) / 2
        want = float((grads[i].double() * step.double()).sum())
        size = float((grads[i].double().norm() * step.double().norm()))
        # third-order terms: (0.02)^2 of a slope of the directions' size; rounding of the outputs far below
        assert abs(slope - want) <= 5e-3 * size, (i, slope, want, size)


@pytest.mark.parametrize("dtype", TYPES)
def test_slices_and_expanded_gradients(dtype):
    T, tol = TYPES[dtype]
    gen = torch.Generator().manual_seed(11)
    B, L, H, Hk, dk, dv = 2, 70, 4, 2, 24, 40
    for off in (0, 1):
        p = (torch.randn(B, L, off + Hk * 2 * dk + H * dv, generator=gen) * 0.2).to(T).to(DEV)
        gb = torch.rand(B, L, 2 * H + 1, generator=gen).to(DEV)
        q, k, v = p[..., off:].split([Hk * dk, Hk * dk, H * dv], -1)
        q, k, v = q.unflatten(-1, (Hk, dk)), k.unflatten(-1, (Hk, dk)), v.unflatten(-1, (H, dv))
        do = torch.randn(B, 1, H, dv, generator=gen).to(T).to(DEV).expand(B, L, H, dv)
        check_backward([q, k, v], -gb[..., :H], gb[..., H:2 * H], None, do, None, tol)


def test_the_same_bits_every_time_and_on_another_stream():
    x, g, b, s0, do, ds = make(3, 300, 4, 2, 128, 128, torch.bfloat16, seed=15)
    first = api.delta_backward(*x, g, b, do, s0, ds)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = api.delta_backward(*x, g, b, do, s0, ds)
    torch.cuda.current_stream().wait_stream(side)
    for a, c in zip(first, again):
        assert torch.equal(a, c)


def test_the_workspace_stays_ready_for_the_scans():
    ws = api.new_workspace(1 << 27, DEV)
    gen = torch.Generator().manual_seed(16)
    a, y = (torch.rand(2, 700, 96, generator=gen).to(DEV) for _ in range(2))
    want = api.linscan_diag(a, y)
    x, g, b, s0, do, ds = make(1, 200, 2, 2, 64, 64, torch.bfloat16, seed=17)
    first = api.delta_backward(*x, g, b, do, s0, ds)
    for _ in range(3):
        for t, c in zip(api.delta_backward(*x, g, b, do, s0, ds, ws=ws), first):
            assert torch.equal(t, c)
        assert torch.equal(api.linscan_diag(a, y, ws=ws), want)


def test_refusals():
    x, g, b, s0, do, ds = make(1, 4, 4, 2, 16, 16, torch.float32, seed=18)
    with pytest.raises(ValueError):
        api.delta_backward(*x, g, b, do[:, :3])
    with pytest.raises(TypeError):
        api.delta_backward(*x, g, b, do.bfloat16())
    with pytest.raises(ValueError):
        api.delta_backward(*x, g, b, do, s0, ds[:, :2])
    with pytest.raises(ValueError):
        api.delta_backward(*x, g, b, do, s0, ds, ws=api.new_workspace(1024, DEV))
