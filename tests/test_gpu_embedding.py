"""GPU parity of the embedding lookup (one fp32 product an element: equal to
torch's) and of its gradient.  Gradients of small integers sum exactly, so any
wrong index or missing row shows as an inequality; random ones are held to
64 * 2^-24 = 4e-6 of the 2-norm (fp32) and one rounding, 2^-8 with room, in bf16."""
import pytest
import torch

from nonlinear_rnn_solve_pararnn_amd import api
from tests import lm_ref
from tests.gpu_helpers import DEV, say

pytestmark = pytest.mark.gpu

TYPES = {"f32": (torch.float32, 4e-6), "bf16": (torch.bfloat16, 2.0 ** -8)}


def ids_of(N, V, kind, seed, dtype=torch.int64):
    gen = torch.Generator().manual_seed(seed)
    if kind == "uniform":
        ids = torch.randint(0, V, (N,), generator=gen)
    elif kind == "same":
        ids = torch.full((N,), V - 1)
    elif kind == "two":
        ids = torch.randint(0, 2, (N,), generator=gen) * (V - 1)
    else:  # the r-th most frequent about 1/r
        u = torch.rand(N, generator=gen, dtype=torch.float64)
        ids = (torch.exp(u * torch.log(torch.tensor(float(V)))).long() - 1).clamp(0, V - 1)
    return ids.to(dtype).to(DEV)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("N,V,D", [(1, 1, 1), (3, 5, 7), (64, 100, 64), (65, 1000, 100), (1000, 300, 257), (129, 70, 1032),
                                   (5000, 50000, 16), (33, 20, 4096)])
def test_lookup(N, V, D, dtype):
    T, _ = TYPES[dtype]
    gen = torch.Generator().manual_seed(N + D)
    table = torch.randn(V, D, generator=gen).to(T).to(DEV)
    for it in (torch.int64, torch.int32):
        ids = ids_of(N, V, "uniform", N, it)
        want = (table.float()[ids.long()] * 2.7).to(T)
        assert torch.equal(api.embedding_forward(ids, table, scale=2.7), want)
    if N == 64:
        assert api.embedding_forward(ids.view(8, 8), table).shape == (8, 8, D)
        odd = torch.empty(V * D + 1, dtype=T, device=DEV)[1:].view(V, D).copy_(table)
        assert torch.equal(api.embedding_forward(ids, odd, scale=2.7), want)


def test_ids_outside_the_table():
    table = torch.ones(10, 32, device=DEV)
    ids = torch.tensor([3, -1, 10, 1 << 40, 9, -(1 << 40)], device=DEV)
    out = api.embedding_forward(ids, table)
    bad = torch.tensor([False, True, True, True, False, True], device=DEV)
    assert torch.isnan(out[bad]).all() and torch.equal(out[~bad], torch.ones(2, 32, device=DEV))
    grad = api.embedding_backward(ids, torch.ones(6, 32, device=DEV), 10)
    want = torch.zeros(10, 32, device=DEV)
    want[3] = want[9] = 1
    assert torch.equal(grad, want)


# one and two sort passes, the one-workgroup sort's edge, chunk edges, wide and odd rows
GRADS = [(1, 1, 1), (5, 3, 7), (16, 255, 64), (17, 256, 64), (300, 2, 100), (1000, 70000, 40), (2000, 500, 257),
         (8192, 300, 24), (8193, 300, 24), (16384, 1000, 8), (16400, 5000, 72), (40000, 33000, 16), (70000, 65, 33)]


@pytest.mark.parametrize("kind", ["uniform", "frequent", "same", "two"])
@pytest.mark.parametrize("N,V,D", GRADS)
def test_gradient_of_integers_is_exact(N, V, D, kind):
    gen = torch.Generator().manual_seed(N)
    grad = torch.randint(-8, 9, (N, D), generator=gen).float().to(DEV)
    ids = ids_of(N, V, kind, N + 1)
    want = torch.zeros(V, D, dtype=torch.float64).index_add_(0, ids.cpu(), grad.cpu().double())
    say("embedding gradient", N, V, D, kind)
    out = torch.full((V, D), float("nan"), device=DEV)  # every row is written
    got = api.embedding_backward(ids, grad, V, scale=2.0, out=out)
    assert got is out and torch.equal(got.cpu().double(), 2.0 * want)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("N,V,D", [(100, 40, 33), (3000, 1000, 256), (9000, 2000, 64)])
def test_gradient_of_random_values(N, V, D, dtype):
    T, tol = TYPES[dtype]
    gen = torch.Generator().manual_seed(D)
    grad = torch.randn(N, D, generator=gen).to(T).to(DEV)
    for it in (torch.int64, torch.int32):
        ids = ids_of(N, V, "frequent", D, it)
        want = lm_ref.embedding_grad(ids.cpu(), grad.cpu().double(), V, 1.5, padding_idx=0)
        got = api.embedding_backward(ids, grad, V, scale=1.5, padding_idx=0)
        e = lm_ref.rel(got, want)
        say(N, V, D, dtype, e)
        assert e <= tol and not got[0].any()
        for _ in range(2):
            assert torch.equal(api.embedding_backward(ids, grad, V, scale=1.5, padding_idx=0), got)


def test_gradient_of_a_larger_vocabulary_takes_three_passes():
    ids = torch.tensor([70000, 199999, 70000, 65536, 0, 131072, 0], device=DEV)
    grad = torch.arange(1.0, 8.0, device=DEV)[:, None].expand(7, 5).contiguous()
    for n in (1, 2000):  # one workgroup's sort, and the longer one
        got = api.embedding_backward(ids.repeat(n), grad.repeat(n, 1), 200000)
        want = torch.zeros(200000, 5, device=DEV)
        want[70000], want[199999], want[65536], want[0], want[131072] = 4.0 * n, 2.0 * n, 4.0 * n, 12.0 * n, 6.0 * n
        assert torch.equal(got, want)


def test_not_finite_gradients_stay_in_their_row():
    ids = ids_of(500, 40, "uniform", 3)
    grad = torch.ones(500, 64, device=DEV)
    grad[123] = float("nan")
    bad = int(ids[123])
    got = api.embedding_backward(ids, grad, 40)
    rows = torch.arange(40, device=DEV) != bad
    assert torch.isnan(got[bad]).all() and torch.isfinite(got[rows]).all()


def test_refusals():
    table, ids = torch.zeros(10, 8, device=DEV), torch.zeros(4, dtype=torch.int64, device=DEV)
    with pytest.raises(TypeError):
        api.embedding_forward(ids.float(), table)
    with pytest.raises(ValueError):
        api.embedding_forward(ids.cpu(), table)
    with pytest.raises(ValueError):
        api.embedding_forward(ids, table[0])
    with pytest.raises(api.PararnnError):
        api.embedding_forward(ids[:0], table)
    with pytest.raises(ValueError):
        api.embedding_backward(ids, torch.zeros(3, 8, device=DEV), 10)
    with pytest.raises(ValueError):
        api.embedding_backward(ids, torch.zeros(4, 8, device=DEV), 10, padding_idx=10)
    with pytest.raises(api.PararnnError):
        api.embedding_backward(ids, torch.zeros(4, 8, device=DEV), 0)
