"""Autograd wiring of the delta-rule mixer on the CPU: the library's calls are
replaced by the fp64 references (tests/mixer_ref.py) and the gradients compared
with torch's autograd through the same formulas; refusals that need no GPU."""
import ctypes

import pytest
import torch

from nonlinear_rnn_solve_pararnn_amd import api, sequence
from tests import mixer_ref as ref
from tests.test_sequence import _rand, _same


@pytest.fixture
def plain(monkeypatch):
    def delta_backward(q, k, v, g, b, do, state=None, grad_state=None, *, scale=None, want_state=None):
        out = ref.delta_grads(q, k, v, g, b, do, state, grad_state, scale)
        return (*out[:5], out[5] if want_state else None)

    def where(q, positions):
        return torch.arange(q.shape[1]).expand(q.shape[:2]) if positions is None else positions

    def headnorm_forward(q, k=None, wq=None, wk=None, table=None, positions=None, *, kind="rms", eps=1e-6,
                         interleaved=False):
        out = []
        for x, w in ((q, wq), (k, wk)):
            out.append((None, None) if x is None else ref.headnorm(x, w, table, where(q, positions), kind, eps, interleaved))
        return out[0][0], out[1][0], out[0][1], out[1][1]

    def headnorm_backward(q, k, rq, rk, gq, gk, wq=None, wk=None, table=None, positions=None, *, kind="rms",
                          interleaved=False):
        out = []
        for x, r, g, w in ((q, rq, gq, wq), (k, rk, gk, wk)):
            dx, dw = (None, None) if x is None else ref.headnorm_grads(x, r, g, w, table, where(q, positions), kind, interleaved)
            out.append((dx, dw if w is not None else None))
        return out[0][0], out[1][0], out[0][1], out[1][1]

    monkeypatch.setattr(api, "delta_forward", lambda q, k, v, g, b, state=None, *, scale=None:
                        ref.delta(q, k, v, g, b, state, scale))
    monkeypatch.setattr(api, "delta_backward", delta_backward)
    monkeypatch.setattr(api, "headnorm_forward", headnorm_forward)
    monkeypatch.setattr(api, "headnorm_backward", headnorm_backward)


def test_gated_delta(plain):
    g, b = -torch.rand(2, 5, 4, dtype=torch.float64), torch.rand(2, 5, 4, dtype=torch.float64)
    args = [_rand(2, 5, 2, 3, seed=1), _rand(2, 5, 2, 3, seed=2), _rand(2, 5, 4, 4, seed=3), g, b, _rand(2, 4, 3, 4, seed=4)]
    _same(lambda *a: sequence.gated_delta(*a, scale=0.7), lambda *a: ref.delta(*a, 0.7), args)
    _same(lambda *a: sequence.gated_delta(*a)[0], lambda *a: ref.delta(*a)[0], args[:5])
    _same(lambda *a: sequence.gated_delta(*a)[1], lambda *a: ref.delta(*a)[1] + 0 * a[0].sum(), args[:5])


@pytest.mark.parametrize("kind,interleaved", [("rms", False), ("l2", True)])
def test_head_norm(plain, kind, interleaved):
    q, k, w = _rand(2, 5, 4, 6, seed=1), _rand(2, 5, 2, 6, seed=2), _rand(6, seed=3)
    tab, pos = ref.table(9, 4), torch.randint(0, 9, (2, 5), generator=torch.Generator().manual_seed(4))
    one = lambda x, w: ref.headnorm(x, w, tab, pos, kind, 1e-6, interleaved)[0]  # noqa: E731
    kw = {"kind": kind, "interleaved": interleaved}
    _same(lambda q, k, a, b: sequence.head_norm(q, k, a, b, tab, pos, **kw), lambda q, k, a, b: (one(q, a), one(k, b)), [q, k, w, w + 1])
    _same(lambda q, k: sequence.head_norm(q, k, None, None, tab, pos, **kw)[1], lambda q, k: one(k, None) + 0 * q.sum(), [q, k])
    _same(lambda q, a: sequence.head_norm(q, None, a, None, tab, pos, **kw)[0], one, [q, w])


def test_rotary_table():
    t = sequence.rotary_table(50, 6)
    assert t.shape == (50, 6) and t.dtype == torch.float32
    assert torch.equal(t, ref.table(50, 6).float())
    for bad in ((0, 4), (4, 3), (4, 0)):
        with pytest.raises(ValueError):
            sequence.rotary_table(*bad)


def test_modules_are_their_formulas(plain):
    torch.manual_seed(0)
    m = sequence.GatedDelta(8, 4, 3, 5, key_heads=2).double()
    x, s0 = _rand(2, 6, 8, seed=5), _rand(2, 4, 3, 5, seed=6)

    def formula(x, s0, qkv, gates, out, a, bias, norm):
        q, k, v = (x @ qkv.T).split([6, 6, 20], -1)
        q, k = (t.unflatten(-1, (2, 3)) for t in (q, k))
        q, k = (t * ((t * t).sum(-1, keepdim=True) + 1e-6) ** -0.5 for t in (q, k))
        z = (x @ gates.T).float().to(x.dtype)  # the gates are worked out in fp32
        b, g = torch.sigmoid(z[..., :4]), -torch.exp(a) * torch.log1p(torch.exp(z[..., 4:] + bias))
        o, s = ref.delta(q, k, v.unflatten(-1, (4, 5)), g, b, s0)
        o = o * ((o * o).sum(-1, keepdim=True) / 5 + 1e-6) ** -0.5 * norm
        return o.flatten(2) @ out.T, s

    got, want = m(x, s0), formula(x, s0, *(p.detach() for p in (m.qkv, m.gates, m.out, m.a, m.bias, m.norm)))
    for a, b in zip(got, want):
        assert float((a - b).detach().norm() / b.norm()) < 1e-6  # fp32 gates in both
    # every parameter gets a gradient
    (got[0].sum() + got[1].sum()).backward()
    assert all(p.grad is not None and bool(p.grad.abs().sum() > 0) for p in m.parameters())


def test_module_arguments():
    for bad in (lambda: sequence.GatedDelta(8, 2, 257), lambda: sequence.GatedDelta(8, 2, 1), lambda: sequence.GatedDelta(8, 3, 4, key_heads=2),
                lambda: sequence.LinearAttention(8, 2, 4, norm="max"), lambda: sequence.LinearAttention(8, 2, 4, rotary=2),
                lambda: sequence.LinearAttention(8, 2, 4, norm="l2", rotary=3), lambda: sequence.LinearAttention(8, 2, 4, norm="rms", rotary=6)):
        with pytest.raises(ValueError):
            bad()
    m = sequence.GatedDelta(8, 2, 4)
    with pytest.raises(ValueError):
        m(torch.zeros(2, 8))
    with pytest.raises(ValueError):
        m.step(torch.zeros(2, 3, 8), None)
    plain = sequence.LinearAttention(8, 2, 4)
    assert len(list(plain.parameters())) == 2 and set(plain.state_dict()) == {"qkv", "out", "log_decay"}
    with pytest.raises(ValueError):
        plain(torch.zeros(1, 2, 8), None, torch.zeros(1, 2, dtype=torch.long))


# ---------------------------------------------------------------- the C ABI's refusals (before any launch)
@pytest.fixture(scope="module")
def lib():
    return api.load_library()


def test_workspace_queries(lib):
    ws = lib.pararnn_delta_workspace_bytes
    for back in (0, 1):
        assert ws(back, 0, 2, 100, 4, 2, 64, 64) > 256
        assert ws(back, 2, 2, 100, 4, 2, 64, 64) == 0      # no such type
        assert ws(back, 0, 2, 100, 4, 3, 64, 64) == 0      # heads that do not divide
        assert ws(back, 0, 2, 100, 4, 0, 64, 64) == 0
        assert ws(back, 0, 0, 100, 4, 4, 64, 64) == 0
        assert ws(back, 0, 2, 100, 4, 4, 257, 64) == 0
        assert ws(back, 0, 1, 1 << 40, 4, 4, 64, 64) == 0
        assert ws(back, 1, 1 << 23, 1, 2, 2, 64, 64) == 0
    assert ws(0, 0, 1, 1 << 26, 1, 1, 64, 64) > 0 and ws(1, 0, 1, (1 << 27) - 32, 1, 1, 64, 64) > 0
    assert ws(1, 0, 1, 1 << 27, 1, 1, 64, 64) == 0
    hw = lib.pararnn_headnorm_workspace_bytes
    assert hw(2, 100, 4, 2, 64) > 256 and hw(2, 100, 4, 0, 64) > 256
    assert hw(2, 100, 0, 2, 64) == 0 and hw(2, 100, 4, 2, 1) == 0 and hw(2, 100, 4, 2, 257) == 0 and hw(1 << 14, 1 << 14, 1, 0, 64) == 0


def test_invalid_calls_are_refused_on_the_host(lib):
    """Addresses that no launch may reach: every call is refused before one."""
    A = 1 << 40  # 256-byte aligned, never dereferenced
    arr = lambda *v: (ctypes.c_int64 * len(v))(*v)  # noqa: E731
    f = lambda dt=0, B=1, L=4, H=2, Hk=2, dk=8, dv=8, q=A, st=None, s0=None, so=None, ws=A, n=1 << 30: lib.pararnn_delta_forward(  # noqa: E731
        dt, B, L, H, Hk, dk, dv, q, A, A, A, A, st, s0, 1.0, A, so, ws, n, None)
    unsupported = f(dk=257)
    assert unsupported < 0 and f(dv=300) == unsupported
    bad = f(q=None)
    assert bad < 0 and bad != unsupported
    dense = (64, 16, 8)
    for st in (arr(*dense, *dense, *dense, 8, 2, 1, 8, 2, -1), arr(64, 1 << 22, 8, *dense, *dense, 8, 2, 1, 8, 2, 1)):
        assert f(st=st) == bad
    assert f(dt=5) == f(Hk=0) == f(H=3, Hk=2) == f(ws=None) == f(n=300) == f(ws=A + 16) == f(q=A + 2) == f(B=-1) == f(s0=A, so=A + 64) == bad
    h = lambda d=8, Hk=2, k=A, yk=A, tab=None, P=0, R=0, pos=None, nb=0, kind=0, eps=1e-6: lib.pararnn_headnorm_forward(  # noqa: E731
        0, 1, 4, 2, Hk, d, A, k, None, None, None, tab, P, R, pos, nb, kind, 0, eps, A, yk, None, None, None)
    assert h(d=257) == unsupported
    assert h(d=1) == h(k=None) == h(Hk=0) == h(yk=None) == h(tab=A, P=4, R=3) == h(tab=A, P=4, R=10) == h(tab=A, R=4) == h(R=4, P=4) == bad
    assert h(tab=A, P=4, R=4, pos=A, nb=2) == h(tab=A, P=4, R=4, pos=A + 4, nb=8) == h(kind=2) == h(eps=-1.0) == h(eps=float("nan")) == bad
