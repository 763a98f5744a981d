"""The gated delta rule's single token on the GPU where a state's rows are not
16-byte vectors: widths that are no multiple of 4, states at odd addresses.

Tolerances are those of tests/test_gpu_delta.py.  The time is held to six times
that of the next whole width: single elements take two to four times as long,
and a form that keeps its rows in memory seventy."""
import statistics

import pytest
import torch

from nonlinear_rnn_solve_pararnn_amd import api
from tests import mixer_ref as ref
from tests.gpu_helpers import DEV
from tests.lm_ref import f64, rel
from tests.test_gpu_delta import F32_TOL, TYPES, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dk,dv", [(1, 3), (31, 33), (64, 33), (127, 127), (128, 66), (129, 1), (256, 255)])
def test_widths(dk, dv, dtype):
    T, tol = TYPES[dtype]
    x, g, b, s0, _, _ = make(3, 1, 4, 2, dk, dv, T, seed=dk + dv)
    o, s = api.delta_step(*(t[:, 0] for t in x), g[:, 0], b[:, 0], s0)
    ro, rs = ref.delta(*f64(*x), *f64(g, b, s0))
    assert rel(o, ro[:, 0]) <= tol and rel(s, rs) <= F32_TOL


def test_a_state_that_begins_at_any_element():
    x, g, b, s0, _, _ = make(3, 1, 4, 2, 64, 64, torch.bfloat16, seed=5)
    args = [t[:, 0].contiguous() for t in (*x, g, b)]
    want = api.delta_step(*args, s0)
    buf = torch.empty(2 * s0.numel() + 2, device=DEV)
    here, there = buf[1:s0.numel() + 1].view(s0.shape), buf[s0.numel() + 1:-1].view(s0.shape)
    here.copy_(s0)
    o, s = api.delta_step(*args, here, out_state=there)
    assert rel(o, want[0].double().cpu()) <= 2.0 ** -8 and rel(s, want[1].double().cpu()) <= F32_TOL
    o2, s2 = api.delta_step(*args, here, out_state=here)
    assert torch.equal(o2, o) and torch.equal(s2, s)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dk", (64, 128, 256))
def test_time(dk, dtype):
    def us(dv):
        x, g, b, s0, _, _ = make(64, 1, 16, 16, dk, dv, TYPES[dtype][0], seed=1)
        args = [t[:, 0].contiguous() for t in (*x, g, b)]
        times = []
        for _ in range(15):
            a, c = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            a.record()
            for _ in range(10):
                api.delta_step(*args, s0, out_state=s0)
            c.record()
            c.synchronize()
            times.append(a.elapsed_time(c))
        return statistics.median(times)

    assert us(127) <= 6 * us(128)
