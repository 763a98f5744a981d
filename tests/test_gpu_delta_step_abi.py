"""The C ABI's single token of the gated delta rule on the GPU: strides of
positions are not read."""
import ctypes

import pytest
import torch

from nonlinear_rnn_solve_pararnn_amd import api
from tests.gpu_helpers import DEV
from tests.test_gpu_delta import make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("between", (0, -1, 1 << 22, 1 << 40))
def test_strides_of_positions_are_ignored(between):
    x, g, b, s0, _, _ = make(3, 1, 4, 2, 24, 40, torch.float32, seed=60)
    q, k, v, g, b = (t[:, 0].contiguous() for t in (*x, g, b))
    want = api.delta_step(q, k, v, g, b, s0)
    strides = []
    for t in (q, k, v, g, b):
        strides += [t.stride(0), between, t.stride(1)]
    o, s = torch.empty_like(v), torch.empty_like(s0)
    at = lambda t: t.data_ptr()  # noqa: E731
    status = api.load_library().pararnn_delta_step(0, 3, 4, 2, 24, 40, at(q), at(k), at(v), at(g), at(b),
                                                   (ctypes.c_int64 * 15)(*strides), at(s0), 24 ** -0.5, at(o), at(s),
                                                   torch.cuda.current_stream().cuda_stream)
    assert status == 0
    assert torch.equal(o, want[0]) and torch.equal(s, want[1])


def test_a_token_of_a_cache_ordered_by_time():
    """Tokens 2^22 elements and more apart in memory."""
    x, g, b, s0, _, _ = make(2, 1, 2, 2, 64, 64, torch.bfloat16, seed=61)
    q, k, v, g, b = (t[:, 0].contiguous() for t in (*x, g, b))
    cache = torch.zeros(2, 1 << 22, dtype=torch.bfloat16, device=DEV)   # [position, everything of one position]
    n = q.numel()
    for i, t in enumerate((q, k, v)):
        cache[1, i * n:(i + 1) * n] = t.reshape(-1)
    views = [cache[:, i * n:(i + 1) * n].unflatten(1, tuple(q.shape)).transpose(0, 1)[:, 1] for i in range(3)]
    want, got = api.delta_step(q, k, v, g, b, s0), api.delta_step(*views, g, b, s0)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
