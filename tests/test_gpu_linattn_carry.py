"""What linear attention carries along a sequence to which nothing is added
(keys or values of zero, a loss on the final state alone), head by head against
e^(g L) of it in fp64, at decays from slow to strong.

Tolerances, relative in the 2-norm of each head.  Carrying a state over a chunk
rounds its factor and the product, 2 * 2^-24; with at most 32 chunks in these
sequences 64 * 2^-24 = 4e-6, the operator's own.  Outputs and gradients in bf16
as everywhere, 4e-3.  A single token's step rounds its factor and the product
alike, so L of them are within 2 L * 2^-24."""
import math

import pytest
import torch

from nonlinear_rnn_solve_pararnn_amd import api
from tests import lm_ref
from tests.gpu_helpers import DEV, say
from tests.test_gpu_linattn import F32_TOL, TYPES

pytestmark = pytest.mark.gpu

# slow, the modules' first head (7/8), 0.8, and down to e^-1 a position
DECAYS = (-0.02, -0.08, -0.1, math.log(0.875), math.log(0.8), -0.25, -0.5, -1.0, -2.5)


def decays(L):
    """Those under which fp32 still holds what is left after L positions."""
    return torch.tensor([g for g in DECAYS if g * L >= -80.0], dtype=torch.float32)


def inputs(L, dk, dv, dtype, seed):
    g = decays(L)
    H = len(g)
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    x = [t.to(dtype).to(DEV) for t in (r(1, L, H, dk), r(1, L, H, dk), r(1, L, H, dv))]
    return x, g.to(DEV), r(1, H, dk, dv).to(DEV)


def heads_rel(got, ref, dim):
    return max(lm_ref.rel(a, b) for a, b in zip(got.unbind(dim), ref.unbind(dim)))


# one short chunk, one whole, several with a short last one, chunks of 64 in bf16, several segments
LENGTHS = [5, 20, 32, 64, 77, 200, 256, 300, 1000]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("zero", ["keys", "values"])
@pytest.mark.parametrize("L", LENGTHS)
def test_state_under_nothing_new(L, zero, dtype):
    T, tol = TYPES[dtype]
    (q, k, v), g, s0 = inputs(L, 64, 48, T, seed=L)
    (k if zero == "keys" else v).zero_()
    o, s = api.linattn_forward(q, k, v, g, s0, scale=1.0)
    qd, gd, sd = lm_ref.f64(q, g, s0)
    want = torch.exp(gd * L).view(1, -1, 1, 1) * sd
    left = torch.exp(gd[None, :] * torch.arange(1, L + 1, dtype=torch.float64)[:, None])
    want_o = torch.einsum("blhi,hij->blhj", qd, sd[0]) * left[None, :, :, None]
    es, eo = heads_rel(s, want, 1), heads_rel(o, want_o, 2)
    say("nothing new", L, zero, dtype, es, eo)
    assert es <= F32_TOL and eo <= tol, (es, eo)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("L", LENGTHS)
def test_loss_on_the_final_state_alone(L, dtype):
    T, tol = TYPES[dtype]
    (q, k, v), g, ds = inputs(L, 48, 64, T, seed=L + 1)
    _, gk, gv, gs = api.linattn_backward(q, k, v, g, torch.zeros_like(v), torch.zeros_like(ds), ds, scale=1.0)
    kd, vd, gd, dd = lm_ref.f64(k, v, g, ds)
    left = torch.exp(gd[None, :] * torch.arange(L - 1, -1, -1, dtype=torch.float64)[:, None])[None, :, :, None]
    errs = (heads_rel(gk, torch.einsum("blhj,hij->blhi", vd, dd[0]) * left, 2),
            heads_rel(gv, torch.einsum("blhi,hij->blhj", kd, dd[0]) * left, 2),
            heads_rel(gs, torch.exp(gd * L).view(1, -1, 1, 1) * dd, 1))
    say("loss on the final state", L, dtype, errs)
    assert errs[0] <= tol and errs[1] <= tol and errs[2] <= F32_TOL, errs


@pytest.mark.parametrize("dtype", TYPES)
def test_prompt_of_zero_keys_agrees_with_single_tokens(dtype):
    T, _ = TYPES[dtype]
    L = 64
    (q, k, v), g, s0 = inputs(L, 32, 40, T, seed=3)
    k.zero_()
    _, s = api.linattn_forward(q, k, v, g, s0)
    t = s0
    for i in range(L):
        _, t = api.linattn_step(q[:, i], k[:, i], v[:, i], g, t)
    e = heads_rel(s, t.cpu().double(), 1)
    say("prompt and tokens", dtype, e)
    assert e <= F32_TOL + 2 * L * 2.0 ** -24


def test_fresh_values_at_strong_decays():
    """The same heads with something to add at every position: the recurrence in fp64."""
    L = 300
    g = torch.tensor(DECAYS, device=DEV)
    gen = torch.Generator().manual_seed(4)
    q, k, v = (torch.randn(1, L, len(DECAYS), 32, generator=gen).to(DEV) for _ in range(3))
    o, s = api.linattn_forward(q, k, v, g)
    ro, rs = lm_ref.linattn(*lm_ref.f64(q, k, v, g))
    assert heads_rel(o, ro, 2) <= F32_TOL and heads_rel(s, rs, 1) <= F32_TOL
