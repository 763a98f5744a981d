"""GPU parity of linear attention with a decay per head (forward, gradients,
single token) against the fp64 recurrence.

Tolerances, relative in the 2-norm.  fp32: an output is a sum of some hundred
products, each step rounding by at most 2^-24 of a partial sum no larger than
a few times the result's rms: 64 * 2^-24 = 4e-6.  bf16 results: rounding a
result to 8 bits is off by at most 2^-9 of it; two roundings of intermediate
operands, of at most 2^-9 each, are allowed beside it: 3 * 2^-9 = 6e-3 at the
worst, 4e-3 as a root of squares with room.  States are fp32 in both."""
import pytest
import torch

from nonlinear_rnn_solve_pararnn_amd import api
from tests import lm_ref
from tests.gpu_helpers import DEV, say

pytestmark = pytest.mark.gpu

F32_TOL, BF16_TOL = 4e-6, 4e-3
TYPES = {"f32": (torch.float32, F32_TOL), "bf16": (torch.bfloat16, BF16_TOL)}


def make(B, L, H, dk, dv, dtype, seed, state=True):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    x = [t.to(dtype).to(DEV) for t in (r(B, L, H, dk), r(B, L, H, dk) * dk ** -0.5, r(B, L, H, dv))]
    g = -torch.exp2(-1.0 - 8.0 * torch.rand(H, generator=gen)).to(DEV)
    s0 = r(B, H, dk, dv).to(DEV) if state else None
    return x, g, s0, r(B, L, H, dv).to(dtype).to(DEV), r(B, H, dk, dv).to(DEV) if state else None


def check_forward(x, g, s0, tol, **kw):
    o, s = api.linattn_forward(*x, g, s0, **kw)
    ro, rs = lm_ref.linattn(*lm_ref.f64(*x), *lm_ref.f64(g, s0), scale=kw.get("scale"))
    eo, es = lm_ref.rel(o, ro), lm_ref.rel(s, rs)
    say("forward", tuple(x[0].shape), x[2].shape[-1], x[0].dtype, eo, es)
    assert o.dtype == x[0].dtype and s.dtype == torch.float32
    assert eo <= tol and es <= F32_TOL, (eo, es)
    return o, s


def check_backward(x, g, s0, do, ds, tol, **kw):
    got = api.linattn_backward(*x, g, do, s0, ds, want_state=True, **kw)
    ref = lm_ref.linattn_grads(*lm_ref.f64(*x), *lm_ref.f64(g, do, s0, ds), scale=kw.get("scale"))
    errs = [lm_ref.rel(a, b) for a, b in zip(got, ref)]
    say("backward", tuple(x[0].shape), x[2].shape[-1], x[0].dtype, errs)
    assert max(errs[:3]) <= tol and errs[3] <= F32_TOL, errs
    return got


# lengths around the chunk, one position, head sizes around the tiles, odd sizes
SHAPES = [(1, 1, 1, 1, 1), (2, 3, 2, 8, 8), (1, 31, 2, 16, 16), (1, 32, 3, 64, 64), (2, 33, 9, 20, 70),
          (1, 64, 2, 128, 128), (1, 65, 2, 128, 64), (3, 127, 5, 48, 80), (1, 130, 1, 65, 129), (2, 100, 3, 17, 33),
          (1, 200, 2, 256, 256), (1, 97, 1, 200, 8), (1, 40, 1, 8, 200), (2, 513, 2, 32, 96)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("B,L,H,dk,dv", SHAPES)
def test_forward_and_backward(B, L, H, dk, dv, dtype):
    T, tol = TYPES[dtype]
    x, g, s0, do, ds = make(B, L, H, dk, dv, T, seed=L * 7 + dk)
    check_forward(x, g, s0, tol)
    check_backward(x, g, s0, do, ds, tol)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("L,H,dk,dv", [(4099, 1, 64, 128), (2500, 3, 128, 40), (3000, 2, 33, 31)])
def test_long_sequence_with_few_rows(L, H, dk, dv, dtype):
    T, tol = TYPES[dtype]
    x, g, s0, do, ds = make(1, L, H, dk, dv, T, seed=L)
    check_forward(x, g, s0, tol)
    check_backward(x, g, s0, do, ds, tol)


@pytest.mark.parametrize("dtype", TYPES)
def test_without_states(dtype):
    T, tol = TYPES[dtype]
    x, g, _, do, _ = make(2, 150, 3, 64, 64, T, seed=5, state=False)
    check_forward(x, g, None, tol)
    check_backward(x, g, None, do, None, tol)
    o, s = api.linattn_forward(*x, g, want_state=False)
    assert s is None
    assert api.linattn_backward(*x, g, do)[3] is None


@pytest.mark.parametrize("dtype", TYPES)
def test_scale_and_extreme_decays(dtype):
    """No decay, a decay that forgets within a position, minus infinity, and one that needs all its bits."""
    T, tol = TYPES[dtype]
    x, _, s0, do, ds = make(1, 300, 4, 64, 48, T, seed=6)
    for g in ([0.0, -1e-6, -0.01, -0.5], [-8.0, -60.0, -1000.0, 0.0]):
        g = torch.tensor(g, device=DEV)
        check_forward(x, g, s0, tol, scale=0.3)
        check_backward(x, g, s0, do, ds, tol, scale=0.3)
    g = torch.tensor([float("-inf"), 0.0, -0.1, float("-inf")], device=DEV)
    o, s = api.linattn_forward(*x, g, s0, scale=1.0)
    q, k, v = (t.double() for t in x)
    for h in (0, 3):  # only the position itself is left
        only = (q[:, :, h] * k[:, :, h]).sum(-1, keepdim=True) * v[:, :, h]
        assert lm_ref.rel(o[:, :, h], only.cpu()) <= tol
        assert lm_ref.rel(s[:, h], (k[:, -1, h, :, None] * v[:, -1, h, None, :]).cpu()) <= F32_TOL


@pytest.mark.parametrize("dtype", TYPES)
def test_small_integers_are_exact(dtype):
    """Without decay every product and sum of small integers is exact, so every index shows."""
    T, _ = TYPES[dtype]
    gen = torch.Generator().manual_seed(7)
    B, L, H, dk, dv = 2, 75, 3, 40, 72
    q, k, v, do = (torch.randint(-1, 2, s, generator=gen).to(T).to(DEV)
                   for s in ((B, L, H, dk), (B, L, H, dk), (B, L, H, dv), (B, L, H, dv)))
    g = torch.zeros(H, device=DEV)
    s0 = torch.randint(-2, 3, (B, H, dk, dv), generator=gen).float().to(DEV)
    o, s = api.linattn_forward(q, k, v, g, s0, scale=1.0)
    ro, rs = lm_ref.linattn(*lm_ref.f64(q, k, v, g, s0), scale=1.0)
    assert torch.equal(s.cpu().double(), rs)
    grads = api.linattn_backward(q, k, v, g, do, s0, s0, scale=1.0)
    refs = lm_ref.linattn_grads(*lm_ref.f64(q, k, v, g, do, s0, s0), scale=1.0)
    assert torch.equal(grads[3].cpu().double(), refs[3])
    if dtype == "f32":
        for a, b in zip((o, *grads[:3]), (ro, *refs[:3])):
            assert torch.equal(a.cpu().double(), b)


@pytest.mark.parametrize("dtype", TYPES)
def test_strided_operands(dtype):
    """One packed projection [B, L, H, dk + dk + dv], heads before positions, a shared key head, and an offset that
    breaks the 16-byte alignment."""
    T, tol = TYPES[dtype]
    (q, k, v), g, s0, do, ds = make(2, 90, 4, 32, 64, T, seed=8)
    packed = torch.cat([q, k, v], -1)
    x = packed.split([32, 32, 64], -1)
    assert not x[0].is_contiguous()
    check_forward(x, g, s0, tol)
    check_backward(x, g, s0, do, ds, tol)
    x = [t.transpose(1, 2).contiguous().transpose(1, 2) for t in (q, k, v)]
    got = check_backward(x, g, s0, do.transpose(1, 2).contiguous().transpose(1, 2), ds, tol)
    assert all(t.is_contiguous() for t in got)
    check_forward([q, k[:, :, :1].expand(-1, -1, 4, -1), v[:, :, :1].expand(-1, -1, 4, -1)], g, s0, tol)
    odd = [torch.empty(t.numel() + 1, dtype=T, device=DEV)[1:].view(t.shape).copy_(t) for t in (q, k, v)]
    a, b = check_forward(odd, g, s0, tol)
    c, d = api.linattn_forward(q, k, v, g, s0)
    assert lm_ref.rel(a, c.cpu().double()) <= tol and torch.equal(b, d)


def test_gradient_matches_differences():
    """The loss is linear in q, k, v and state, each alone: a difference over a
    whole step is the gradient's product with it, to fp32 rounding."""
    x, g, s0, do, ds = make(1, 70, 2, 32, 48, torch.float32, seed=9)
    grads = api.linattn_backward(*x, g, do, s0, ds)

    def loss(q, k, v, s):
        o, S = api.linattn_forward(q, k, v, g, s)
        return float((o.double() * do).sum() + (S.double() * ds).sum())

    args = [*x, s0]
    base = loss(*args)
    for i, grad in enumerate(grads):
        step = torch.randn(grad.shape, generator=torch.Generator().manual_seed(i)).to(DEV)
        moved = list(args)
        moved[i] = args[i] + step
        want = float((grad.double() * step).sum())
        size = float(grad.double().norm() * step.double().norm())
        # both losses sum thousands of fp32 results of this size
        assert abs((loss(*moved) - base) - want) <= 1e-5 * (size + abs(base)), (i, want)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("where", ["q", "k", "v"])
def test_not_finite_values_stay_behind(where, dtype):
    """A NaN or infinity at position t leaves every earlier output as it was (and for the gradients, what it cannot reach)."""
    T, _ = TYPES[dtype]
    x, g, s0, do, ds = make(1, 100, 2, 32, 64, T, seed=10)
    clean, _ = api.linattn_forward(*x, g, s0)
    for bad in (float("nan"), float("inf")):
        y = [t.clone() for t in x]
        y["qkv".index(where)][0, 41, 0, 3] = bad
        o, s = api.linattn_forward(*y, g, s0)
        assert torch.equal(o[:, :41], clean[:, :41])
        assert torch.equal(o[:, :, 1], clean[:, :, 1])
        assert not torch.isfinite(o[0, 41, 0]).all()
        assert torch.isfinite(s[0, 1]).all() and (where == "q") == bool(torch.isfinite(s[0, 0]).all())
        if where == "q":
            assert torch.equal(o[:, 42:], clean[:, 42:])
    if where == "v":  # dv, dk of later positions come from positions after them alone
        y = do.clone()
        y[0, 41, 0, 3] = float("nan")
        a = api.linattn_backward(*x, g, do, s0, ds)
        b = api.linattn_backward(*x, g, y, s0, ds)
        assert torch.equal(a[0][:, :41], b[0][:, :41]) and torch.equal(a[0][:, 42:], b[0][:, 42:])
        for i in (1, 2):
            assert torch.equal(a[i][:, 42:], b[i][:, 42:])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("B,H,dk,dv", [(1, 1, 1, 1), (3, 5, 16, 16), (2, 7, 48, 80), (1, 16, 128, 128), (5, 3, 33, 31),
                                       (2, 2, 256, 256), (1, 3, 7, 130), (64, 16, 64, 64)])
def test_single_token(B, H, dk, dv, dtype):
    T, tol = TYPES[dtype]
    x, g, s0, _, _ = make(B, 1, H, dk, dv, T, seed=dk * 3 + dv)
    y = [t[:, 0] for t in x]
    o, s = api.linattn_step(*y, g, s0)
    ro, rs = lm_ref.linattn(*lm_ref.f64(*x), *lm_ref.f64(g, s0))
    eo, es = lm_ref.rel(o, ro[:, 0]), lm_ref.rel(s, rs)
    say("step", B, H, dk, dv, dtype, eo, es)
    assert eo <= tol and es <= F32_TOL
    s1 = s0.clone()
    o1, same = api.linattn_step(*y, g, s1, out_state=s1)
    assert same is s1 and torch.equal(s1, s) and torch.equal(o1, o)
    packed = torch.cat(y, -1)
    o2, s2 = api.linattn_step(*packed.split([dk, dk, dv], -1), g, s0)
    assert torch.equal(o2, o) and torch.equal(s2, s)


@pytest.mark.parametrize("dtype", TYPES)
def test_prompt_then_tokens_equals_the_whole(dtype):
    T, tol = TYPES[dtype]
    x, g, s0, _, _ = make(2, 75, 3, 64, 64, T, seed=11)
    whole, final = api.linattn_forward(*x, g, s0)
    o, s = api.linattn_forward(*[t[:, :70] for t in x], g, s0)
    rows = [o]
    for t in range(70, 75):
        o, s = api.linattn_step(*[y[:, t] for y in x], g, s, out_state=s)
        rows.append(o[:, None])
    assert lm_ref.rel(torch.cat(rows, 1), whole.cpu().double()) <= tol
    assert lm_ref.rel(s, final.cpu().double()) <= F32_TOL
    # the state may be continued in place
    s = s0.clone()
    api.linattn_forward(*x, g, s, out_state=s)
    assert torch.equal(s, final)


def test_same_bits_every_time_and_on_another_stream():
    x, g, s0, do, ds = make(2, 700, 3, 64, 64, torch.bfloat16, seed=12)
    a = (*api.linattn_forward(*x, g, s0), *api.linattn_backward(*x, g, do, s0, ds))
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        b = (*api.linattn_forward(*x, g, s0), *api.linattn_backward(*x, g, do, s0, ds))
    torch.cuda.current_stream().wait_stream(st)
    for p, q in zip(a, b):
        assert torch.equal(p, q)


def test_workspace_is_shared_with_the_scans():
    """The scans' records and this operator's scratch take turns in one workspace."""
    ws = api.new_workspace(64 << 20, DEV)
    gen = torch.Generator().manual_seed(13)
    a, b = torch.rand(2, 3000, 40, generator=gen).to(DEV), torch.randn(2, 3000, 40, generator=gen).to(DEV)
    x, g, s0, do, ds = make(1, 2000, 1, 64, 64, torch.float32, seed=13)
    h = api.linscan_diag(a, b, ws=ws)
    o, s = api.linattn_forward(*x, g, s0, ws=ws)
    for _ in range(3):
        assert torch.equal(api.linscan_diag(a, b, ws=ws), h)
        assert torch.equal(api.linattn_forward(*x, g, s0, ws=ws)[0], o)
        api.linattn_backward(*x, g, do, s0, ds, ws=ws)


def test_refusals():
    x, g, s0, do, _ = make(1, 8, 2, 16, 16, torch.float32, seed=14)
    q, k, v = x
    for bad in ((q, k[:, :4], v), (q, k, v[:, :, :1]), (q, k[..., :8], v)):
        with pytest.raises(ValueError):
            api.linattn_forward(*bad, g)
    with pytest.raises(TypeError):
        api.linattn_forward(q, k.bfloat16(), v, g)
    with pytest.raises(TypeError):
        api.linattn_forward(q, k, v, g.double())
    with pytest.raises(ValueError):
        api.linattn_forward(q, k, v, g[:1])
    with pytest.raises(ValueError):
        api.linattn_forward(q, k, v, g, s0[..., :8])
    with pytest.raises(ValueError, match="dense"):
        api.linattn_forward(q, torch.empty(1, 8, 2, 32, device=DEV)[..., ::2], v, g)
    with pytest.raises(api.PararnnError):
        api.linattn_forward(q[:, :0], k[:, :0], v[:, :0], g)
    with pytest.raises(api.PararnnError, match="head sizes"):
        y = torch.zeros(1, 8, 2, 257, device=DEV)
        api.linattn_forward(y, y, v, g)
    with pytest.raises(ValueError):
        api.linattn_forward(q[0], k[0], v[0], g)
    with pytest.raises(ValueError):
        api.linattn_backward(q, k, v, g, do[:, :3])
    with pytest.raises(ValueError):
        api.linattn_forward(q, k, v, g, ws=torch.zeros(16, dtype=torch.uint8, device=DEV))
