"""Layer norm with more rows than a launch takes at once, so that every
workgroup goes round several times and the last round is not full, and gradients
written over what they are computed from.  Tolerances of
tests/test_gpu_layernorm.py; rows of 3 elements with eps 0.1, as without it the
rows whose elements nearly agree are rounding error in any fp32 form."""
import pytest
import torch

from nonlinear_rnn_solve_pararnn_amd import api
from tests.gpu_helpers import DEV
from tests.test_gpu_layernorm import TYPES, check, make

pytestmark = pytest.mark.gpu

# 16 lanes, a wave, a workgroup a row in registers; rows read several times; a lane a row (backward)
SHAPES = [(16500, 64), (40001, 100), (4099, 256), (9001, 513), (5003, 1000), (2063, 1028), (1025, 4099), (1030, 8192),
          (2100, 8200)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("R,D", SHAPES)
def test_several_rounds(R, D, dtype):
    T, tol = TYPES[dtype]
    x, r, w, b, dy, ds = make(R, D, T, seed=R + D)
    check(x, w, b, r, dy, ds, tol)
    check(x, None, None, None, dy, None, tol)


@pytest.mark.parametrize("dtype", TYPES)
def test_several_rounds_of_three_elements(dtype):
    T, tol = TYPES[dtype]
    x, r, w, b, dy, ds = make(140000, 3, T, seed=3)
    check(x, w, b, r, dy, ds, tol, eps=0.1)
    check(x, None, None, None, dy, None, tol, eps=0.1)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("over", ["grad_y", "grad_sum"])
@pytest.mark.parametrize("R,D", [(3000, 3), (9, 3), (5000, 100), (5000, 1000), (1500, 1283), (1100, 4096), (300, 8200),
                                 (7, 20001)])
def test_gradient_written_over_an_input(R, D, over, dtype):
    T, _ = TYPES[dtype]
    lib = api.load_library()
    x, _, w, _, dy, ds = make(R, D, T, seed=R + D + 1)
    _, s, mean, rstd = api.layernorm_forward(x, w)
    want = api.layernorm_backward(s, w, mean, rstd, dy, ds)
    gy, gs = dy.clone(), ds.clone()
    dx = gy if over == "grad_y" else gs
    gw, gb = torch.empty_like(w), torch.empty_like(w)
    ws = torch.zeros(lib.pararnn_layernorm_workspace_bytes(R, D), dtype=torch.uint8, device=DEV)
    at = lambda t: t.data_ptr()  # noqa: E731
    status = lib.pararnn_layernorm_backward(0 if dtype == "f32" else 1, R, D, at(s), at(w), at(mean), at(rstd), at(gy), at(gs),
                                            at(dx), at(gw), at(gb), at(ws), ws.numel(),
                                            torch.cuda.current_stream().cuda_stream)
    assert status == 0
    assert torch.equal(dx, want[0]) and torch.equal(gw, want[1]) and torch.equal(gb, want[2])
