"""GPU parity of the norms of queries and keys for each head with the position
rotation (forward, gradients) against the fp64 formulas.

Tolerances, relative in the 2-norm.  fp32: an element is a product of four or
five numbers rounded by 2^-24 each, of which r carries a sum of up to 256
squares (8 roundings of partial sums in a chain of vectors and lanes, half of
which r's square root keeps): 16 * 2^-24 = 1e-6.  bf16 results are rounded once
from fp32, each by 2^-8 of the value at the most, so their 2-norm is off by at
most 2^-8 of it and what the fp32 values are off by (a root of squares over many
elements is 2^-8 / sqrt(3), but tensors here have as few as three): 2^-8 +
1e-6.  Weight gradients are sums of many rows in fp32: 64 * 2^-24 = 4e-6."""
import pytest
import torch

from nonlinear_rnn_solve_pararnn_amd import api
from tests import mixer_ref as ref
from tests.gpu_helpers import DEV, say
from tests.lm_ref import f64, rel

pytestmark = pytest.mark.gpu

F32_TOL, SUM_TOL = 1e-6, 4e-6
BF16_TOL = 2.0 ** -8 + F32_TOL
TYPES = {"f32": (torch.float32, F32_TOL), "bf16": (torch.bfloat16, BF16_TOL)}


def make(B, L, Hq, Hk, d, R, dtype, seed, weight=True, P=None):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    P = L + 50 if P is None else P
    x = [(t * 2).to(dtype).to(DEV) for t in (r(B, L, Hq, d), r(B, L, Hk, d))]
    dy = [t.to(dtype).to(DEV) for t in (r(B, L, Hq, d), r(B, L, Hk, d))]
    w = [(1 + 0.2 * r(d)).to(DEV) for _ in range(2)] if weight else [None, None]
    tab = ref.table(P, R).float().to(DEV) if R else None
    pos = torch.randint(0, P, (B, L), generator=gen).to(DEV) if R else None
    return x, dy, w, tab, pos


def check(x, dy, w, tab, pos, tol, kind, interleaved, eps=1e-6):
    got = api.headnorm_forward(*x, *w, tab, pos, kind=kind, eps=eps, interleaved=interleaved)
    where = pos
    if tab is not None and pos is None:
        where = torch.arange(x[0].shape[1], device=DEV).expand(x[0].shape[:2])
    tab64, pos64 = (None, None) if tab is None else (tab.cpu().double(), where.cpu().long())
    errs = []
    for i in range(2):
        y, r = ref.headnorm(*f64(x[i], w[i]), tab64, pos64, kind, eps, interleaved)
        errs += [rel(got[i], y), rel(got[2 + i], r)]
        assert got[i].dtype == x[i].dtype and got[2 + i].dtype == torch.float32
    back = api.headnorm_backward(*x, got[2], got[3], *dy, *w, tab, pos, kind=kind, interleaved=interleaved)
    sums = []
    for i in range(2):
        dx, dw = ref.headnorm_grads(*f64(x[i], got[2 + i], dy[i], w[i]), tab64, pos64, kind, interleaved)
        errs.append(rel(back[i], dx))
        if w[i] is not None:
            sums.append(rel(back[2 + i], dw))
        else:
            assert back[2 + i] is None
    say("headnorm", tuple(x[0].shape), x[1].shape[2], x[0].dtype, kind, interleaved, errs, sums)
    assert max(errs[1], errs[3]) <= F32_TOL and max(errs) <= tol, errs
    assert not sums or max(sums) <= SUM_TOL, sums
    return got, back


# sizes around the 16 lanes' vectors, odd ones, one element, partial rotations that cross vectors
SHAPES = [(1, 1, 1, 1, 3, 0), (2, 3, 4, 2, 2, 2), (1, 5, 3, 1, 16, 16), (2, 7, 16, 4, 64, 64), (1, 33, 5, 5, 65, 64),
          (3, 17, 16, 16, 128, 64), (1, 9, 2, 1, 130, 100), (2, 4, 3, 3, 256, 256), (1, 50, 8, 2, 40, 16), (1, 6, 1, 9, 96, 34),
          (2, 300, 16, 8, 128, 128)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("B,L,Hq,Hk,d,R", SHAPES)
@pytest.mark.parametrize("kind,interleaved", [("rms", False), ("l2", True)])
def test_forward_and_backward(B, L, Hq, Hk, d, R, kind, interleaved, dtype):
    T, tol = TYPES[dtype]
    check(*make(B, L, Hq, Hk, d, R, T, seed=d * 3 + R), tol, kind, interleaved)


@pytest.mark.parametrize("dtype", TYPES)
def test_without_weights_and_positions(dtype):
    T, tol = TYPES[dtype]
    x, dy, w, tab, _ = make(2, 60, 6, 3, 64, 32, T, seed=1, weight=False)
    check(x, dy, w, tab, None, tol, "rms", False)
    check(x, dy, [w[0], torch.ones(64, device=DEV)], None, None, tol, "l2", False)


def test_one_tensor_and_one_token():
    x, dy, w, tab, pos = make(3, 4, 6, 2, 48, 48, torch.bfloat16, seed=2)
    both = api.headnorm_forward(*x, *w, tab, pos)
    alone = api.headnorm_forward(x[0], None, w[0], None, tab, pos)
    assert torch.equal(alone[0], both[0]) and torch.equal(alone[2], both[2]) and alone[1] is None and alone[3] is None
    gb = api.headnorm_backward(*x, both[2], both[3], *dy, *w, tab, pos)
    ga = api.headnorm_backward(x[0], None, alone[2], None, dy[0], None, w[0], None, tab, pos)
    assert torch.equal(ga[0], gb[0]) and rel(ga[2], gb[2].double().cpu()) < SUM_TOL and ga[1] is None and ga[3] is None
    one = api.headnorm_forward(x[0][:, 1], x[1][:, 1], *w, tab, pos[:, 1].contiguous())
    assert torch.equal(one[0], both[0][:, 1]) and torch.equal(one[1], both[1][:, 1])


@pytest.mark.parametrize("dtype", TYPES)
def test_slices_of_a_projection(dtype):
    """Strided views, at any alignment, against the formulas (other alignments add a row's squares up in another order)."""
    T, tol = TYPES[dtype]
    gen = torch.Generator().manual_seed(3)
    for off, pad in ((0, 3), (1, 3), (8, 0), (8, 8)):
        p = torch.randn(2, 9, pad + 6 * 64 + off, generator=gen).to(T).to(DEV)
        q, k = p[..., off:off + 256].unflatten(-1, (4, 64)), p[..., off + 256:off + 384].unflatten(-1, (2, 64))
        dy = [torch.randn(*t.shape, generator=gen).to(T).to(DEV) for t in (q, k)]
        check([q, k], dy, [None, None], ref.table(9, 64).float().to(DEV), None, tol, "rms", False)


def test_rows_of_zeros_and_values_that_are_not_finite():
    x, dy, w, tab, pos = make(1, 4, 3, 2, 32, 16, torch.float32, seed=4)
    x[0][0, 0] = 0.0
    x[0][0, 1, 1, 3] = float("nan")
    x[0][0, 2, 2, 20] = float("inf")
    y, _, r, _ = api.headnorm_forward(*x, *w, tab, pos, eps=1e-6)
    assert torch.equal(y[0, 0], torch.zeros_like(y[0, 0])) and torch.allclose(r[0, 0], torch.full_like(r[0, 0], 1e3), rtol=1e-6)
    bad = torch.zeros(1, 4, 3, dtype=torch.bool, device=DEV)
    bad[0, 1, 1] = bad[0, 2, 2] = True
    assert bool((torch.isfinite(y).all(-1) == ~bad).all())


@pytest.mark.parametrize("bits", [torch.int32, torch.int64])
def test_positions_outside_the_table(bits):
    x, dy, w, tab, _ = make(1, 5, 3, 2, 32, 16, torch.float32, seed=5, P=40)
    pos = torch.tensor([[0, 39, 40, -1, 2 ** 31 - 1]], device=DEV).to(bits)
    y, _, r, rk = api.headnorm_forward(*x, *w, tab, pos)
    fine = torch.isfinite(y)
    assert bool(fine[:, :2].all()) and not bool(fine[:, 2:, :, :16].any()) and bool(fine[:, 2:, :, 16:].all())
    same = api.headnorm_forward(*x, *w, tab, pos[:, :].clamp(0, 39))[0]
    assert torch.equal(same[:, :2], y[:, :2]) and torch.equal(same[..., 16:], y[..., 16:])


def test_the_same_bits_every_time_and_on_another_stream():
    x, dy, w, tab, pos = make(2, 700, 16, 4, 128, 128, torch.bfloat16, seed=6)
    first = api.headnorm_forward(*x, *w, tab, pos)
    gfirst = api.headnorm_backward(*x, first[2], first[3], *dy, *w, tab, pos)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = api.headnorm_forward(*x, *w, tab, pos)
        gagain = api.headnorm_backward(*x, again[2], again[3], *dy, *w, tab, pos)
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(first + gfirst, again + gagain):
        assert torch.equal(a, b)


def test_refusals():
    x, dy, w, tab, pos = make(1, 4, 2, 2, 32, 16, torch.float32, seed=7)
    with pytest.raises(TypeError):
        api.headnorm_forward(x[0].half(), x[1])
    with pytest.raises(TypeError):
        api.headnorm_forward(x[0], x[1].bfloat16())
    with pytest.raises(ValueError):
        api.headnorm_forward(x[0], x[1], kind="max")
    with pytest.raises(ValueError):
        api.headnorm_forward(x[0], x[1][:, :3])
    with pytest.raises(ValueError):
        api.headnorm_forward(x[0], x[1], None, None, tab[:, :15].contiguous(), pos)
    with pytest.raises(ValueError):
        api.headnorm_forward(x[0], x[1], None, None, tab[:3].contiguous())
    with pytest.raises(ValueError):
        api.headnorm_forward(x[0], x[1], None, None, None, pos)
    with pytest.raises(ValueError):
        api.headnorm_forward(x[0][:, 0], x[1][:, 0], None, None, tab)
    with pytest.raises(ValueError):
        api.headnorm_forward(x[0], None, None, w[1])
    with pytest.raises(api.PararnnError):
        api.headnorm_forward(torch.zeros(1, 1, 1, 257, device=DEV))
    with pytest.raises(api.PararnnError):
        api.headnorm_forward(torch.zeros(1, 1, 1, 1, device=DEV))
    with pytest.raises(api.PararnnError):
        api.headnorm_forward(torch.zeros(1, 0, 1, 8, device=DEV))
    with pytest.raises(api.PararnnError):
        api.headnorm_forward(x[0], x[1], eps=-1.0)
