"""Linear attention on operands that lie inside larger allocations: what is
before the first and after the last position belongs to others and reaches no
result, whatever it holds.  Against the fp64 recurrence, with the tolerances of
tests/test_gpu_linattn.py (the same sums of products)."""
import pytest
import torch

from nonlinear_rnn_solve_pararnn_amd import api
from tests import lm_ref
from tests.gpu_helpers import DEV, say
from tests.test_gpu_linattn import F32_TOL, TYPES, make

pytestmark = pytest.mark.gpu

NAN = float("nan")


def inside(t, shift, heads_first):
    """A copy of t [B, L, H, d] that begins `shift` elements after a 16-byte
    aligned place, NaN in everything around it; heads before positions if asked."""
    room = torch.full((t.numel() + 64,), NAN, dtype=t.dtype, device=DEV)
    n = 16 // t.element_size() + shift
    src = t.transpose(1, 2) if heads_first else t
    dst = room[n:n + t.numel()].view(src.shape).copy_(src)
    return dst.transpose(1, 2) if heads_first else dst


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("B,L,H,dk,dv,heads_first", [
    (1, 333, 1, 77, 77, False), (2, 333, 3, 77, 77, True), (1, 333, 1, 64, 64, False), (2, 45, 3, 64, 33, True),
    (1, 1, 1, 1, 1, False), (1, 13, 1, 9, 130, False), (1, 1101, 2, 101, 31, True)])
@pytest.mark.parametrize("shift", [0, 1, 2, 7])
def test_neighbours_reach_nothing(B, L, H, dk, dv, heads_first, shift, dtype):
    T, tol = TYPES[dtype]
    x, g, s0, do, ds = make(B, L, H, dk, dv, T, seed=L + dk)
    ro, rs = lm_ref.linattn(*lm_ref.f64(*x), *lm_ref.f64(g, s0))
    refs = lm_ref.linattn_grads(*lm_ref.f64(*x), *lm_ref.f64(g, do, s0, ds))
    *y, dy = (inside(t, shift, heads_first) for t in (*x, do))
    o, s = api.linattn_forward(*y, g, s0)
    grads = api.linattn_backward(*y, g, dy, s0, ds)
    errs = [lm_ref.rel(a, b) for a, b in zip((o, s, *grads), (ro, rs, *refs))]
    say("neighbours", B, L, H, dk, dv, heads_first, shift, dtype, errs)
    assert all(t.isfinite().all() for t in (o, s, *grads))
    assert errs[1] <= F32_TOL and errs[5] <= F32_TOL and max(errs[:1] + errs[2:5]) <= tol, errs


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("d", [33, 64, 77])
def test_heads_of_one_tensor_do_not_meet(d, dtype):
    """Heads before positions: the next head's first element follows this head's last one."""
    T, _ = TYPES[dtype]
    x, g, s0, do, ds = make(1, 333, 3, d, d, T, seed=d)
    y = [inside(t, 1, True) for t in (*x, do)]
    clean = (*api.linattn_forward(*y[:3], g, s0), *api.linattn_backward(*y[:3], g, y[3], s0, ds))
    for t in y:
        t[0, 0, 1, 0] = t[0, -1, 1, -1] = NAN
    got = (*api.linattn_forward(*y[:3], g, s0), *api.linattn_backward(*y[:3], g, y[3], s0, ds))
    for i, (a, b) in enumerate(zip(got, clean)):
        heads = 2 if a.shape[1] == 333 else 1
        pick = torch.tensor([0, 2], device=DEV)
        assert torch.equal(a.index_select(heads, pick), b.index_select(heads, pick)), i


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("step", [0, 1, 8])
def test_rows_that_overlap(step, dtype):
    """Windows of one sequence: position t is the elements from step t on."""
    T, tol = TYPES[dtype]
    L, d = 77, 64
    (q, k, _), g, s0, _, _ = make(1, L, 1, d, d, T, seed=step + 20)
    flat = torch.randn(step * (L - 1) + d, generator=torch.Generator().manual_seed(step)).to(T).to(DEV)
    v = flat.as_strided((1, L, 1, d), (flat.numel(), step, d, 1))
    o, s = api.linattn_forward(q, k, v, g, s0)
    ro, rs = lm_ref.linattn(*lm_ref.f64(q, k, v, g, s0))
    assert lm_ref.rel(o, ro) <= tol and lm_ref.rel(s, rs) <= F32_TOL
    if step:
        flat[-1] = NAN  # the last position's last element alone
        p, _ = api.linattn_forward(q, k, v, g, s0)
        assert torch.equal(p[:, :-1], o[:, :-1]) and p[0, -1, 0, -1].isnan()
        p, r = api.linattn_forward(q, v, k, g, s0)
        w, _ = api.linattn_forward(q, v.nan_to_num(0.0), k, g, s0)
        assert torch.equal(p[:, :-1], w[:, :-1]) and r[0, 0, :-1].isfinite().all() and r[0, 0, -1].isnan().all()
