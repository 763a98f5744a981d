"""Autograd wiring of sequence.py on the CPU: the library's calls are replaced
by the fp64 references (tests/lm_ref.py) and the gradients compared with
torch's autograd through the same formulas."""
import pytest
import torch

from nonlinear_rnn_solve_pararnn_amd import api, sequence
from tests import lm_ref


@pytest.fixture
def plain(monkeypatch):
    def linattn_forward(q, k, v, g, state=None, *, scale=None):
        return lm_ref.linattn(q, k, v, g, state, scale)

    def linattn_backward(q, k, v, g, do, state=None, grad_state=None, *, scale=None, want_state=None):
        out = lm_ref.linattn_grads(q, k, v, g, do, state, grad_state, scale)
        return (*out[:3], out[3] if want_state else None)

    def layernorm_forward(x, w=None, b=None, residual=None, *, eps=1e-5):
        s = x if residual is None else x + residual
        y, mean, rstd = lm_ref.layernorm(s, w, b, eps)
        return y, s, mean, rstd

    def layernorm_backward(s, w, mean, rstd, dy, ds=None, *, want_w=True, want_b=True):
        dx, dw, db = lm_ref.layernorm_grads(s, w, mean, rstd, dy, ds)
        return dx, dw if want_w else None, db if want_b else None

    monkeypatch.setattr(api, "linattn_forward", linattn_forward)
    monkeypatch.setattr(api, "linattn_backward", linattn_backward)
    monkeypatch.setattr(api, "layernorm_forward", layernorm_forward)
    monkeypatch.setattr(api, "layernorm_backward", layernorm_backward)
    monkeypatch.setattr(api, "embedding_forward", lambda ids, table, *, scale=1.0: table[ids] * scale)
    monkeypatch.setattr(api, "embedding_backward", lambda ids, g, V, *, scale=1.0, padding_idx=None:
                        lm_ref.embedding_grad(ids, g, V, scale, padding_idx))


def _rand(*shape, seed=0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed), dtype=torch.float64)


def _same(fn, ref, args, seed=50):
    """Gradients of a random combination of fn's outputs equal those of ref's."""
    outs = []
    for f in (fn, ref):
        ts = [a.clone().requires_grad_(True) for a in args]
        got = f(*ts)
        got = got if isinstance(got, tuple) else (got,)
        loss = sum((o * _rand(*o.shape, seed=seed + i)).sum() for i, o in enumerate(got))
        outs.append([*got, *torch.autograd.grad(loss, ts)])
    for a, b in zip(*outs):
        assert lm_ref.rel(a, b.detach()) < 1e-12


def test_linear_attention(plain):
    g = -torch.rand(3, dtype=torch.float64)
    args = [_rand(2, 6, 3, 4, seed=1), _rand(2, 6, 3, 4, seed=2), _rand(2, 6, 3, 5, seed=3), _rand(2, 3, 4, 5, seed=4)]
    _same(lambda q, k, v, s: sequence.linear_attention(q, k, v, g, s, scale=0.7),
          lambda q, k, v, s: lm_ref.linattn(q, k, v, g, s, 0.7), args)
    _same(lambda q, k, v: sequence.linear_attention(q, k, v, g)[0], lambda q, k, v: lm_ref.linattn(q, k, v, g)[0], args[:3])
    _same(lambda q, k, v: sequence.linear_attention(q, k, v, g)[1], lambda q, k, v: lm_ref.linattn(q, k, v, g)[1] + 0 * q.sum(),
          args[:3])
    # a key head shared by all heads gets the sum of their gradients
    one = args[1][:, :, :1]
    _same(lambda q, k, v: sequence.linear_attention(q, k.expand(-1, -1, 3, -1), v, g)[0],
          lambda q, k, v: lm_ref.linattn(q, k.expand(-1, -1, 3, -1), v, g)[0], [args[0], one, args[2]])


def test_layer_norm(plain):
    x, r, w, b = _rand(4, 5, 6, seed=1), _rand(4, 5, 6, seed=2), _rand(6, seed=3), _rand(6, seed=4)
    ref = lambda x, w, b, r: (lm_ref.layernorm(x + r, w, b)[0], x + r)  # noqa: E731
    _same(lambda x, w, b, r: sequence.layer_norm(x, w, b, r), ref, [x, w, b, r])
    _same(lambda x, w, b: sequence.layer_norm(x, w, b), lambda x, w, b: ref(x, w, b, torch.zeros_like(x)), [x, w, b])
    _same(lambda x, w, b: sequence.layer_norm(x, w, b)[0], lambda x, w, b: lm_ref.layernorm(x, w, b)[0], [x, w, b])
    _same(lambda x, r: sequence.layer_norm(x, None, None, r)[1], lambda x, r: x + r, [x, r])


def test_embedding(plain):
    ids = torch.tensor([[0, 3, 3], [1, 0, 4]])
    _same(lambda t: sequence.embedding(ids, t, scale=1.5), lambda t: t[ids] * 1.5, [_rand(6, 4)])
    t = _rand(6, 4).requires_grad_(True)
    sequence.embedding(ids, t, padding_idx=3).sum().backward()
    assert not t.grad[3].any() and t.grad[0].eq(2).all()


def test_no_second_derivative_and_no_decay_gradient(plain):
    q = _rand(1, 3, 2, 4).requires_grad_(True)
    g = torch.zeros(2, dtype=torch.float64)
    o, _ = sequence.linear_attention(q, q.detach(), q.detach(), g)
    (first,) = torch.autograd.grad(o.sum(), q, create_graph=True)
    with pytest.raises(RuntimeError):
        torch.autograd.grad(first.sum(), q)
    with pytest.raises(ValueError, match="constant"):
        sequence.linear_attention(q, q, q, g.requires_grad_(True))


def test_module_arguments():
    for bad in (lambda: sequence.LinearAttention(8, 2, 257), lambda: sequence.LinearAttention(8, 0, 4),
                lambda: sequence.LinearAttention(8, 2, 4, log_decay=torch.zeros(3)), lambda: sequence.LayerNorm(0),
                lambda: sequence.LayerNorm(4, eps=float("nan")), lambda: sequence.Embedding(4, 8, padding_idx=4)):
        with pytest.raises(ValueError):
            bad()
    m = sequence.LinearAttention(8, 2, 4)
    assert "log_decay" in m.state_dict() and len(list(m.parameters())) == 2
    with pytest.raises(ValueError):
        m(torch.zeros(2, 8))
    with pytest.raises(ValueError):
        m.step(torch.zeros(2, 3, 8), None)
