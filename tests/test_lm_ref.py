"""The fp64 references of the operators around the recurrences against torch's
autograd and against differences (CPU), and the binding's refusals that need
no GPU."""
import ctypes

import pytest
import torch

from nonlinear_rnn_solve_pararnn_amd import api
from tests import lm_ref


def _inputs(B=2, L=7, H=3, dk=4, dv=5, seed=0):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)  # noqa: E731
    g = -torch.rand(H, generator=gen, dtype=torch.float64)
    return r(B, L, H, dk), r(B, L, H, dk), r(B, L, H, dv), g, r(B, H, dk, dv), r(B, L, H, dv), r(B, H, dk, dv)


def test_linattn_gradients_match_autograd():
    q, k, v, g, s0, do, ds = _inputs()
    ts = [t.clone().requires_grad_(True) for t in (q, k, v, s0)]
    o, S = lm_ref.linattn(*ts[:3], g, ts[3])
    want = torch.autograd.grad((o * do).sum() + (S * ds).sum(), ts)
    for a, b in zip(lm_ref.linattn_grads(q, k, v, g, do, s0, ds), want):
        assert lm_ref.rel(a, b) < 1e-12


def test_linattn_gradients_match_differences():
    """The loss is linear in each of q, k, v and state alone, so a difference
    over any step is the gradient's product with it."""
    q, k, v, g, s0, do, ds = _inputs(seed=1)

    def loss(q, k, v, s0):
        o, S = lm_ref.linattn(q, k, v, g, s0)
        return float((o * do).sum() + (S * ds).sum())

    grads = lm_ref.linattn_grads(q, k, v, g, do, s0, ds)
    args = [q, k, v, s0]
    base = loss(*args)
    for i, grad in enumerate(grads):
        step = torch.randn(grad.shape, generator=torch.Generator().manual_seed(i), dtype=torch.float64)
        moved = list(args)
        moved[i] = args[i] + step
        assert abs((loss(*moved) - base) - float((grad * step).sum())) < 1e-9 * (1 + abs(base))


def test_layernorm_gradients_match_autograd_and_differences():
    gen = torch.Generator().manual_seed(2)
    s, w, b, dy, ds = (torch.randn(*n, generator=gen, dtype=torch.float64) for n in ((6, 9), (9,), (9,), (6, 9), (6, 9)))
    ts = [t.clone().requires_grad_(True) for t in (s, w, b)]

    def loss(s, w, b):
        return (lm_ref.layernorm(s, w, b)[0] * dy).sum() + (s * ds).sum()

    want = torch.autograd.grad(loss(*ts), ts)
    _, mean, rstd = lm_ref.layernorm(s, w, b)
    got = lm_ref.layernorm_grads(s, w, mean, rstd, dy, ds)
    for x, y in zip(got, want):
        assert lm_ref.rel(x, y) < 1e-12
    step = torch.randn(6, 9, generator=gen, dtype=torch.float64)
    h = 1e-5
    diff = float(loss(s + h * step, w, b) - loss(s - h * step, w, b)) / (2 * h)
    assert abs(diff - float((got[0] * step).sum())) < 1e-7 * (1 + abs(diff))


def test_embedding_gradient_matches_autograd():
    gen = torch.Generator().manual_seed(3)
    table = torch.randn(11, 4, generator=gen, dtype=torch.float64, requires_grad=True)
    ids = torch.randint(0, 11, (3, 8), generator=gen)
    grad = torch.randn(3, 8, 4, generator=gen, dtype=torch.float64)
    (want,) = torch.autograd.grad((table[ids] * 2.5 * grad).sum(), table)
    assert lm_ref.rel(lm_ref.embedding_grad(ids, grad, 11, 2.5), want) < 1e-12


# ---------------------------------------------------------------- refusals on the host
@pytest.fixture(scope="module")
def lib():
    return api.load_library()


def test_library_refuses_invalid_arguments(lib):
    """Checked before any device call: the pointers below are never used."""
    n, f, one = None, ctypes.c_void_p(0x10000), ctypes.c_float(1.0)
    big = 1 << 30
    args = lambda dt, B, L, H, dk, dv, q=f: (dt, B, L, H, dk, dv, q, f, f, n, f, n, one, f, n, f, big, n)  # noqa: E731
    assert lib.pararnn_linattn_forward(*args(0, 0, 4, 4, 8, 8)) == -1
    assert lib.pararnn_linattn_forward(*args(2, 1, 4, 4, 8, 8)) == -1            # type
    assert lib.pararnn_linattn_forward(*args(0, 1, 4, 4, 0, 8)) == -1
    assert lib.pararnn_linattn_forward(*args(0, 1, 4, 4, 257, 8)) == -3          # head size
    assert lib.pararnn_linattn_forward(*args(0, 1, 4, 4, 8, 257)) == -3
    assert lib.pararnn_linattn_forward(*args(0, 1, 4, 4, 8, 8, n)) == -1         # null operand
    assert lib.pararnn_linattn_forward(*args(0, 1, 4, 4, 8, 8, ctypes.c_void_p(0x10002))) == -1  # half an fp32 element
    bad = (ctypes.c_int64 * 9)(*([8] * 8 + [-8]))
    assert lib.pararnn_linattn_forward(0, 1, 4, 4, 8, 8, f, f, f, bad, f, n, one, f, n, f, big, n) == -1
    assert lib.pararnn_linattn_forward(0, 1, 4, 4, 8, 8, f, f, f, n, f, n, one, f, n, f, 0, n) == -1     # workspace
    assert lib.pararnn_linattn_forward(0, 1, 4, 4, 8, 8, f, f, f, n, f, n, one, f, n, n, big, n) == -1
    part = ctypes.c_void_p(0x10000 + 4)  # a state that overlaps its successor by all but one element
    assert lib.pararnn_linattn_forward(0, 1, 4, 4, 8, 8, f, f, f, n, f, f, one, f, part, f, big, n) == -1
    assert lib.pararnn_linattn_step(0, 1, 4, 8, 8, f, f, f, n, f, f, one, f, part, n) == -1
    far = (ctypes.c_int64 * 9)(*([64, 1 << 22, 8] * 3))                          # a position's stride
    assert lib.pararnn_linattn_forward(0, 1, 4, 4, 8, 8, f, f, f, far, f, n, one, f, n, f, big, n) == -1
    assert lib.pararnn_linattn_backward(0, 1, 4, 4, 8, 8, f, f, f, n, n, f, n, n, one, f, f, f, n, f, big, n) == -1
    assert lib.pararnn_linattn_step(0, 1, 4, 8, 8, f, f, f, n, f, n, one, f, f, n) == -1                 # no state
    assert lib.pararnn_layernorm_forward(0, 4, 0, f, n, n, n, one, n, f, n, n, n) == -1
    assert lib.pararnn_layernorm_forward(0, 4, 8, f, f, n, n, one, n, f, n, n, n) == -1                  # residual, no sum
    assert lib.pararnn_layernorm_forward(0, 4, 8, f, n, n, n, ctypes.c_float(-1.0), n, f, n, n, n) == -1
    assert lib.pararnn_layernorm_forward(0, 4, 8, f, n, n, n, ctypes.c_float(float("nan")), n, f, n, n, n) == -1
    assert lib.pararnn_layernorm_backward(0, 4, 8, f, n, f, f, f, n, f, f, n, n, 0, n) == -1             # dw, no workspace
    assert lib.pararnn_embedding_forward(0, 4, 8, 8, f, 2, f, one, f, n) == -1                           # id size
    assert lib.pararnn_embedding_forward(0, 0, 8, 8, f, 4, f, one, f, n) == -1
    assert lib.pararnn_embedding_backward(0, 4, 8, 8, f, 4, f, one, 8, f, f, big, n) == -1               # padding_idx
    assert lib.pararnn_embedding_backward(0, 4, 8, 8, f, 4, f, one, -1, f, f, 0, n) == -1


def test_workspace_queries(lib):
    assert lib.pararnn_linattn_workspace_bytes(0, 0, 2, 100, 3, 8, 8) >= 256
    assert lib.pararnn_linattn_workspace_bytes(1, 1, 2, 100, 3, 8, 8) >= 256
    assert lib.pararnn_linattn_workspace_bytes(0, 0, 2, 0, 3, 8, 8) == 0
    assert lib.pararnn_linattn_workspace_bytes(0, 0, 2, 100, 3, 8, 300) == 0
    assert lib.pararnn_layernorm_workspace_bytes(0, 8) == 0
    assert lib.pararnn_embedding_workspace_bytes(1 << 30, 8, 8) == 0
    assert lib.pararnn_embedding_workspace_bytes(100, 8, 8) > 100 * 8


def test_binding_refuses_host_tensors_and_wrong_types():
    x = torch.zeros(2, 4, 3, 8)
    with pytest.raises(ValueError, match="HIP device"):
        api.linattn_forward(x, x, x, torch.zeros(3))
    with pytest.raises(TypeError, match="float32 or bfloat16"):
        api.linattn_forward(x.double(), x.double(), x.double(), torch.zeros(3))
    with pytest.raises(TypeError, match="torch.Tensor"):
        api.layernorm_forward([1.0])
    with pytest.raises(ValueError, match="HIP device"):
        api.layernorm_forward(x)
    with pytest.raises(TypeError, match="float32 or bfloat16"):
        api.embedding_forward(torch.zeros(3, dtype=torch.int64), x.half().view(6, 32))
    with pytest.raises(ValueError, match="HIP device"):
        api.embedding_backward(torch.zeros(3, dtype=torch.int64), torch.zeros(3, 8), 4)
