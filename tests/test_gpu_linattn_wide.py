"""Heads of 129 to 256 over sequences long enough for the longer chunk (bf16,
above 256 positions) and for several segments, against the fp64 recurrence with
the tolerances of tests/test_gpu_linattn.py."""
import pytest
import torch

from tests.gpu_helpers import DEV
from tests.test_gpu_linattn import TYPES, check_backward, check_forward, make

pytestmark = pytest.mark.gpu

# whole walks and segments, 16-byte rows and rows of any alignment, one width narrow
SHAPES = [(1, 600, 2, 256, 256), (1, 2500, 1, 200, 136), (1, 1100, 1, 131, 255), (1, 520, 40, 160, 256),
          (8, 300, 33, 130, 20)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("state", [True, False])
@pytest.mark.parametrize("B,L,H,dk,dv", SHAPES)
def test_wide_heads(B, L, H, dk, dv, state, dtype):
    T, tol = TYPES[dtype]
    x, g, s0, do, ds = make(B, L, H, dk, dv, T, seed=L + dv, state=state)
    check_forward(x, g, s0, tol)
    check_backward(x, g, s0, do, ds, tol)


@pytest.mark.parametrize("dtype", TYPES)
def test_wide_heads_of_a_packed_projection(dtype):
    """Strided views of one tensor, as the modules pass them."""
    T, tol = TYPES[dtype]
    (q, k, v), g, s0, do, ds = make(1, 700, 2, 192, 256, T, seed=2)
    p = torch.cat([t.flatten(2) for t in (q, k, v)], -1).to(DEV)
    x = [t.unflatten(-1, (2, -1)) for t in p.split([2 * 192, 2 * 192, 2 * 256], -1)]
    assert not x[0].is_contiguous()
    check_forward(x, g, s0, tol)
    check_backward(x, g, s0, do, ds, tol)
