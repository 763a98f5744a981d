"""The fp64 references of the delta-rule mixer's operators against torch's
autograd and against differences (CPU)."""
import torch

from tests import mixer_ref as ref
from tests.lm_ref import rel


def _inputs(B=2, L=6, Hk=2, H=4, dk=4, dv=5, seed=0):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)  # noqa: E731
    g, b = -torch.rand(B, L, H, generator=gen, dtype=torch.float64), torch.rand(B, L, H, generator=gen, dtype=torch.float64)
    return [r(B, L, Hk, dk), r(B, L, Hk, dk), r(B, L, H, dv), g, b, r(B, H, dk, dv)], r(B, L, H, dv), r(B, H, dk, dv)


def _loss(q, k, v, g, b, s0, do, ds):
    o, S = ref.delta(q, k, v, g, b, s0)
    return (o * do).sum() + (S * ds).sum()


def test_delta_is_the_formula():
    (q, k, v, g, b, s0), _, _ = _inputs(B=1, L=3, Hk=1, H=1)
    o, S = ref.delta(q, k, v, g, b, s0, scale=2.0)
    T = s0[0, 0]
    eye = torch.eye(4, dtype=torch.float64)
    for t in range(3):
        kt = k[0, t, 0]
        T = torch.exp(g[0, t, 0]) * (eye - b[0, t, 0] * torch.outer(kt, kt)) @ T + b[0, t, 0] * torch.outer(kt, v[0, t, 0])
        assert rel(o[0, t, 0], 2.0 * q[0, t, 0] @ T) < 1e-12
    assert rel(S[0, 0], T) < 1e-12


def test_delta_gradients_match_autograd_and_differences():
    args, do, ds = _inputs()
    ts = [t.clone().requires_grad_(True) for t in args]
    want = torch.autograd.grad(_loss(*ts, do, ds), ts)
    got = ref.delta_grads(*args[:5], do, args[5], ds)
    for a, w in zip(got, want):
        assert rel(a, w) < 1e-12
    h = 1e-6
    for i, grad in enumerate(got):
        step = torch.randn(grad.shape, generator=torch.Generator().manual_seed(i), dtype=torch.float64)
        up, down = list(args), list(args)
        up[i], down[i] = args[i] + h * step, args[i] - h * step
        diff = float(_loss(*up, do, ds) - _loss(*down, do, ds)) / (2 * h)
        # central differences: h^2 times a third derivative of about 1e3, and 1e-16 / h of the loss
        assert abs(diff - float((grad * step).sum())) < 1e-7 * (1 + abs(diff))


def test_headnorm_gradients_match_autograd_and_differences():
    gen = torch.Generator().manual_seed(3)
    r = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)  # noqa: E731
    x, w, dy = r(2, 3, 4, 10), r(10), r(2, 3, 4, 10)
    tab, pos = ref.table(9, 6), torch.tensor([[0, 1, 2], [6, 7, 8]])
    for kind in ("rms", "l2"):
        for interleaved in (False, True):
            def loss(x, w):
                return (ref.headnorm(x, w, tab, pos, kind, 1e-6, interleaved)[0] * dy).sum()
            ts = [t.clone().requires_grad_(True) for t in (x, w)]
            want = torch.autograd.grad(loss(*ts), ts)
            _, rr = ref.headnorm(x, w, tab, pos, kind, 1e-6, interleaved)
            got = ref.headnorm_grads(x, rr, dy, w, tab, pos, kind, interleaved)
            for a, b in zip(got, want):
                # eps in r alone: m(g x r) x r has the same r
                assert rel(a, b) < 1e-12
            h, step = 1e-6, r(2, 3, 4, 10)
            diff = float(loss(x + h * step, w) - loss(x - h * step, w)) / (2 * h)
            assert abs(diff - float((got[0] * step).sum())) < 1e-7 * (1 + abs(diff))


def test_rotation_keeps_lengths_and_turns_by_differences():
    x = torch.randn(1, 5, 1, 8, generator=torch.Generator().manual_seed(4), dtype=torch.float64)
    tab, pos = ref.table(40, 8), torch.arange(5)[None]
    for interleaved in (False, True):
        y = ref.turn(x, tab, pos, interleaved)
        assert rel((y * y).sum(-1), (x * x).sum(-1)) < 1e-12
        assert rel(ref.turn(y, tab, pos, interleaved, back=True), x) < 1e-12
        far = ref.turn(x, tab, pos + 30, interleaved)
        near = lambda z, i, j: (z[0, i, 0] * z[0, j, 0]).sum()  # noqa: E731
        assert abs(near(y, 1, 4) - near(far, 1, 4)) < 1e-12
