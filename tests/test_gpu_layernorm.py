"""GPU parity of layer norm (with the residual sum) and its gradients against
the fp64 formulas.

Tolerances, relative in the 2-norm.  fp32: a few roundings of 2^-24 on each of
y and dx beside the statistics' (sums of D terms in a tree): 32 * 2^-24 = 2e-6;
sums over rows: 64 * 2^-24 = 4e-6.  bf16: one rounding of the result, at most
2^-9 of it: 2^-8 with room.  Statistics, dw and db are fp32 in both."""
import pytest
import torch

from nonlinear_rnn_solve_pararnn_amd import api
from tests import lm_ref
from tests.gpu_helpers import DEV, say

pytestmark = pytest.mark.gpu

TYPES = {"f32": (torch.float32, 2e-6), "bf16": (torch.bfloat16, 2.0 ** -8)}
SUM_TOL = 4e-6
# odd sizes, each register variant and its edge, rows too long for the registers, more rows than workgroups
SHAPES = [(1, 2), (3, 7), (5, 64), (2, 255), (9, 256), (4, 512), (7, 513), (3, 1000), (6, 1024), (5, 1025), (3, 2056),
          (2, 4096), (3, 4100), (2, 8192), (2, 8193), (3, 20000), (9000, 40), (3000, 1028)]


def make(R, D, dtype, seed, shift=0.25):
    gen = torch.Generator().manual_seed(seed)
    x, r, dy, ds = ((torch.randn(R, D, generator=gen) + (shift if i == 0 else 0)).to(dtype).to(DEV) for i in range(4))
    w, b = ((1.0 + 0.2 * torch.randn(D, generator=gen)).to(DEV), (0.2 * torch.randn(D, generator=gen)).to(DEV))
    return x, r, w, b, dy, ds


def check(x, w, b, r, dy, ds, tol, **kw):
    y, s, mean, rstd = api.layernorm_forward(x, w, b, r, **kw)
    if r is None:
        assert s is x
    else:
        assert torch.equal(s, (x.float() + r.float()).to(x.dtype))
    sd, wd, bd, dyd, dsd = lm_ref.f64(s, w, b, dy, ds)
    ry, rm, rr = lm_ref.layernorm(sd, wd, bd, **kw)
    # the mean's own size may be far below the elements it sums
    em = float((mean.cpu().double() - rm).abs().max() / sd.abs().max())
    errs = dict(y=lm_ref.rel(y, ry), mean=em, rstd=lm_ref.rel(rstd, rr))
    dx, dw, db = api.layernorm_backward(s, w, mean, rstd, dy, ds)
    rx, rw, rb = lm_ref.layernorm_grads(sd, wd, *lm_ref.f64(mean, rstd), dyd, dsd)
    errs.update(dx=lm_ref.rel(dx, rx), dw=lm_ref.rel(dw, rw), db=lm_ref.rel(db, rb))
    say("layernorm", tuple(x.shape), x.dtype, errs)
    assert errs["y"] <= tol and errs["dx"] <= tol, errs
    assert errs["mean"] <= 2e-6 and errs["rstd"] <= 2e-6 and errs["dw"] <= SUM_TOL and errs["db"] <= SUM_TOL, errs


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("R,D", SHAPES)
def test_forward_and_backward(R, D, dtype):
    T, tol = TYPES[dtype]
    x, r, w, b, dy, ds = make(R, D, T, seed=R + D)
    check(x, w, b, r, dy, ds, tol)
    check(x, None, None, None, dy, None, tol)


@pytest.mark.parametrize("dtype", TYPES)
def test_unaligned_and_other_layouts(dtype):
    T, tol = TYPES[dtype]
    x, r, w, b, dy, ds = make(12, 512, T, seed=1)
    odd = torch.empty(x.numel() + 1, dtype=T, device=DEV)[1:].view(x.shape).copy_(x)
    check(odd, w, b, r, dy, ds, tol)
    x3 = x.view(3, 4, 512)
    y, s, mean, rstd = api.layernorm_forward(x3, w, b, r.view(3, 4, 512), eps=1e-3)
    assert mean.shape == rstd.shape == (3, 4)
    y2, s2, _, _ = api.layernorm_forward(x, w, b, r, eps=1e-3)
    assert torch.equal(y.view(12, 512), y2) and torch.equal(s.view(12, 512), s2)
    out, tot = torch.empty_like(x), torch.empty_like(x)
    got = api.layernorm_forward(x, w, b, r, eps=1e-3, out=out, out_sum=tot)
    assert got[0] is out and got[1] is tot and torch.equal(out, y2)


def test_large_mean_and_constant_rows():
    """The variance is that of the centred row: a mean a thousand times the
    spread costs about 1000 * 2^-24 * 8 of y, and a constant row gives zeros."""
    x, _, w, b, _, _ = make(6, 1024, torch.float32, seed=2, shift=1000.0)
    y, _, _, _ = api.layernorm_forward(x, w, b)
    ref, _, _ = lm_ref.layernorm(*lm_ref.f64(x, w, b))
    assert lm_ref.rel(y, ref) <= 1000 * 2.0 ** -24 * 8
    c = torch.full((3, 777), 0.5, device=DEV)
    y, _, mean, rstd = api.layernorm_forward(c)
    assert torch.equal(y, torch.zeros_like(c)) and torch.equal(mean, torch.full((3,), 0.5, device=DEV))
    assert float((rstd - 1e-5 ** -0.5).abs().max()) <= 1e-4


def test_not_finite_rows_stay_alone():
    x, r, w, b, dy, ds = make(8, 1024, torch.float32, seed=3)
    clean = api.layernorm_forward(x, w, b)[0]
    x[2, 17], x[5, 0] = float("nan"), float("inf")
    y = api.layernorm_forward(x, w, b)[0]
    keep = [0, 1, 3, 4, 6, 7]
    assert torch.equal(y[keep], clean[keep])
    assert not torch.isfinite(y[2]).any() and not torch.isfinite(y[5]).any()


def test_gradient_matches_differences():
    """Central differences of the forward pass in fp32: y moves by about h, and
    its rounding of 2^-24 a term over h = 2^-6 leaves 1e-5 of the sum's size."""
    x, _, w, b, dy, _ = make(4, 300, torch.float32, seed=4)
    _, s, mean, rstd = api.layernorm_forward(x, w, b)
    dx, dw, db = api.layernorm_backward(s, w, mean, rstd, dy)
    h = 2.0 ** -6
    loss = lambda x, w, b: float((api.layernorm_forward(x, w, b)[0].double() * dy).sum())  # noqa: E731
    for i, (t, g) in enumerate(((x, dx), (w, dw), (b, db))):
        step = torch.randn(t.shape, generator=torch.Generator().manual_seed(i)).to(DEV)
        a = [x, w, b]
        up, dn = list(a), list(a)
        up[i], dn[i] = t + h * step, t - h * step
        diff = (loss(*up) - loss(*dn)) / (2 * h)
        want = float((g.double() * step).sum())
        # the third-order term of the quotient, h^2 of the sum's size, beside the rounding
        assert abs(diff - want) <= (h * h + 1e-4) * float(g.double().norm() * step.double().norm()), (i, diff, want)


def test_partial_gradients_and_repeatability():
    x, r, w, b, dy, ds = make(700, 256, torch.bfloat16, seed=5)
    _, s, mean, rstd = api.layernorm_forward(x, w, b, r)
    a = api.layernorm_backward(s, w, mean, rstd, dy, ds)
    c = api.layernorm_backward(s, w, mean, rstd, dy, ds, want_w=False, want_b=False)
    assert torch.equal(a[0], c[0]) and c[1] is None and c[2] is None
    d = api.layernorm_backward(s, w, mean, rstd, dy, ds, want_w=False)
    assert d[1] is None and torch.equal(d[2], a[2])
    for _ in range(3):
        for p, q in zip(api.layernorm_backward(s, w, mean, rstd, dy, ds), a):
            assert torch.equal(p, q)


def test_refusals():
    x, r, w, b, dy, _ = make(4, 16, torch.float32, seed=6)
    with pytest.raises(ValueError):
        api.layernorm_forward(x, w[:8])
    with pytest.raises(TypeError):
        api.layernorm_forward(x, w.bfloat16())
    with pytest.raises(ValueError, match="contiguous"):
        api.layernorm_forward(x.t())
    with pytest.raises(ValueError):
        api.layernorm_forward(x, residual=r[:2])
    with pytest.raises(ValueError):
        api.layernorm_forward(x, out_sum=r)
    with pytest.raises(api.PararnnError):
        api.layernorm_forward(x[:0])
    with pytest.raises(api.PararnnError):
        api.layernorm_forward(x, eps=-1.0)
    _, s, mean, rstd = api.layernorm_forward(x)
    with pytest.raises(ValueError):
        api.layernorm_backward(s, None, mean[:2], rstd, dy)
    with pytest.raises(TypeError):
        api.layernorm_backward(s, None, mean, rstd, dy.bfloat16())
