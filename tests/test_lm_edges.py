"""Edges of the operators around the recurrences: sizes and overlaps that the
library refuses on the host (CPU), and on the GPU a decay that is not a number,
a gradient written over its input, a state that autograd has saved."""
import ctypes

import pytest
import torch

from nonlinear_rnn_solve_pararnn_amd import api, sequence
from tests import lm_ref
from tests.gpu_helpers import DEV

f, n, one, BIG = ctypes.c_void_p(0x10000), None, ctypes.c_float(1.0), 1 << 40


@pytest.fixture(scope="module")
def lib():
    return api.load_library()


def test_a_launch_holds_the_call(lib):
    """Workgroups of 256 threads, counted in 32 bits: 2^24 of them."""
    query = lib.pararnn_linattn_workspace_bytes
    assert query(0, 0, (1 << 24) - 8, 1, 1, 1, 1) > 0 and query(0, 0, 1 << 24, 1, 1, 1, 1) == 0
    assert query(0, 0, 1 << 22, 1, 1, 1, 256) == 0 and query(0, 0, 1 << 21, 1, 1, 1, 256) > 0
    assert query(1, 0, 1 << 23, 1, 1, 1, 1) == 0 and query(1, 0, 1 << 22, 1, 1, 1, 1) > 0
    assert lib.pararnn_linattn_step(0, 1 << 24, 1, 1, 1, f, f, f, n, f, f, one, f, f, n) == -1
    assert lib.pararnn_embedding_forward(0, 1 << 28, 8, 8, f, 4, f, one, f, n) == -1
    assert lib.pararnn_embedding_workspace_bytes((1 << 28) - 32, 8, 64) > 0
    assert lib.pararnn_embedding_workspace_bytes(1 << 22, 8, 1 << 20) == 0
    assert lib.pararnn_embedding_workspace_bytes(64, 8, (1 << 24) - 1) > 0


def test_state_gradient_stands_alone(lib):
    """The walks that read the states run beside the one that ends on grad_state."""
    a = ctypes.c_void_p(0x10000 + 4 * 8)
    back = lambda s, gs, out: lib.pararnn_linattn_backward(  # noqa: E731
        0, 1, 4, 4, 8, 8, f, f, f, f, n, f, s, gs, one, f, f, f, out, f, BIG, n)
    assert back(f, n, f) == -1 and back(n, f, f) == -1 and back(a, n, f) == -1 and back(n, f, a) == -1


@pytest.mark.gpu
@pytest.mark.parametrize("L", [1, 70, 2000])
def test_decay_that_is_not_a_number(L):
    gen = torch.Generator().manual_seed(L)
    q, k, v, do = (torch.randn(1, L, 3, 32, generator=gen).to(DEV) for _ in range(4))
    g = torch.tensor([-0.1, float("nan"), -0.2], device=DEV)
    o, s = api.linattn_forward(q, k, v, g)
    grads = api.linattn_backward(q, k, v, g, do)
    pick = lambda t: t[:, :, ::2].contiguous()  # noqa: E731
    want_o, want_s = api.linattn_forward(pick(q), pick(k), pick(v), g[::2].contiguous())
    ref_o, ref_s = lm_ref.linattn(*lm_ref.f64(pick(q), pick(k), pick(v), g[::2]))
    assert o[:, :, 1].isnan().all() and s[:, 1].isnan().all()
    assert all(t[:, :, 1].isnan().all() for t in grads[:3])
    assert all(t[:, :, ::2].isfinite().all() for t in grads[:3])
    # 64 roundings of 2^-24, as for every fp32 output of the operator
    assert lm_ref.rel(pick(o), ref_o) <= 4e-6 and lm_ref.rel(s[:, ::2], ref_s) <= 4e-6
    assert lm_ref.rel(want_o, ref_o) <= 4e-6 and lm_ref.rel(want_s, ref_s) <= 4e-6
    o1, s1 = api.linattn_step(q[:, 0], k[:, 0], v[:, 0], g, torch.zeros(1, 3, 32, 32, device=DEV))
    assert o1[:, 1].isnan().all() and s1[:, 1].isnan().all() and o1[:, ::2].isfinite().all()


@pytest.mark.gpu
@pytest.mark.parametrize("D", [3, 1000, 4096, 8200])
def test_norm_gradient_written_over_its_input(D):
    lib = api.load_library()
    gen = torch.Generator().manual_seed(D)
    s, dy = (torch.randn(9, D, generator=gen).to(DEV) for _ in range(2))
    w = torch.randn(D, generator=gen).to(DEV)
    _, _, mean, rstd = api.layernorm_forward(s, w)
    want = api.layernorm_backward(s, w, mean, rstd, dy)
    over, gw, gb = dy.clone(), torch.empty_like(w), torch.empty_like(w)
    ws = torch.zeros(lib.pararnn_layernorm_workspace_bytes(9, D), dtype=torch.uint8, device=DEV)
    at = lambda t: t.data_ptr()  # noqa: E731
    st = lib.pararnn_layernorm_backward(0, 9, D, at(s), at(w), at(mean), at(rstd), at(over), None, at(over), at(gw),
                                        at(gb), at(ws), ws.numel(), torch.cuda.current_stream().cuda_stream)
    assert st == 0
    assert torch.equal(over, want[0]) and torch.equal(gw, want[1]) and torch.equal(gb, want[2])


@pytest.mark.gpu
def test_step_over_a_saved_state_is_noticed():
    mix = sequence.LinearAttention(32, 2, 16, device=DEV)
    state = torch.randn(1, 2, 16, 16, device=DEV)
    x = torch.randn(1, 5, 32, device=DEV)
    y, _ = mix(x, state)
    mix.step(x[:, 0], state)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()
    with torch.inference_mode():
        s = torch.zeros(1, 2, 16, 16, device=DEV)
        mix.step(x[:, 0], s)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("N,D", [(9000, 9), (700, 15), (300, 1031), (33, 518), (2500, 8), (40, 3)])
def test_embedding_rows_that_begin_anywhere(N, D, dtype):
    """Integers small enough that every sum is exact in bf16: groups of columns
    that overlap at a row's end, and tensors that begin inside a word."""
    V = 1200
    gen = torch.Generator().manual_seed(N + D)

    def inside(*shape):
        x = torch.randint(-2, 3, shape, generator=gen).to(dtype)
        flat = torch.empty(x.numel() + 3, dtype=dtype, device=DEV)
        return flat[3:].view(shape).copy_(x)

    ids = torch.randperm(V * 8, generator=gen)[:N].remainder(V)  # at most 8 of one id: sums up to 16
    table, grad, ids = inside(V, D), inside(N, D), ids.to(DEV)
    assert torch.equal(api.embedding_forward(ids, table, scale=2.0), table[ids] * 2)
    out = torch.full((V * D + 8,), 7.0, dtype=dtype, device=DEV)
    got = api.embedding_backward(ids, grad, V, scale=2.0, out=out[5:5 + V * D].view(V, D))
    want = torch.zeros(V, D, dtype=torch.float64).index_add_(0, ids.cpu(), grad.cpu().double()) * 2
    assert torch.equal(got.cpu().double(), want)
    assert (out[:5] == 7).all() and (out[5 + V * D:] == 7).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,D", [(1, 5), (15, 16), (17, 65), (37, 100), (64, 127), (9001, 128), (33, 129)])
def test_norm_of_short_rows(rows, D, dtype):
    """Four rows a wave up to 128 elements, a row each above; tolerances as for every norm."""
    from tests.test_gpu_layernorm import TYPES, check, make
    T, tol = TYPES[dtype]
    x, r, w, b, dy, ds = make(rows, D, T, seed=rows * 3 + D)
    check(x, w, b, r, dy, ds, tol)
    check(x, w, None, None, dy, None, tol)
