"""Edges of the delta-rule mixer's operators on the GPU: sequences in segments
with values that are not finite, states updated in place, wide heads and padded
rows; operands shared, repeated and far apart in memory; two streams at once.

Tolerances are those of the operators' own tests (tests/test_gpu_delta.py,
tests/test_gpu_delta_grads.py); where the same sums run in the same order the
bits are the same."""
import pytest
import torch

from nonlinear_rnn_solve_pararnn_amd import api, sequence
from tests import mixer_ref as ref
from tests.gpu_helpers import DEV
from tests.lm_ref import f64, rel
from tests.test_gpu_delta import BF16_TOL, F32_TOL, check_forward, make
from tests.test_gpu_delta_grads import check_backward

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
TOL = {"f32": (F32_TOL, 1.6e-5), "bf16": (BF16_TOL, 4e-3)}


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("what", ("v", "k", "g", "b", "q"))
def test_values_that_are_not_finite_in_segments(what, dtype):
    x, g, b, s0, _, _ = make(1, 2100, 2, 1, 32, 72, TYPES[dtype], seed=31)
    clean, sclean = api.delta_forward(*x, g, b, s0)
    t = 700
    for value in (float("nan"), float("inf")):
        y, gg, bb = [z.clone() for z in x], g.clone(), b.clone()
        if what in "qkv":
            y["qkv".index(what)][0, t, 0, 5] = value
        else:
            (gg if what == "g" else bb)[0, t, 0] = value
        o, s = api.delta_forward(*y, gg, bb, s0)
        assert torch.equal(o[:, :t], clean[:, :t]), (what, value)
        if what != "q" and what != "k":  # q and k are both heads'
            assert torch.equal(o[:, :, 1], clean[:, :, 1]) and torch.equal(s[:, 1], sclean[:, 1])
        if what == "q":
            assert not bool(torch.isfinite(o[0, t]).any())
            assert torch.equal(o[:, t + 1:], clean[:, t + 1:]) and torch.equal(s, sclean)
        elif what == "v":
            rest = [c for c in range(72) if c != 5]
            assert not bool(torch.isfinite(o[0, t:, 0, 5]).any()) and not bool(torch.isfinite(s[0, 0, :, 5]).any())
            assert torch.equal(o[..., rest], clean[..., rest]) and torch.equal(s[..., rest], sclean[..., rest])
        else:
            assert not bool(torch.isfinite(o[0, t:, 0]).any()) and not bool(torch.isfinite(s[0, 0]).any())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("L,H,Hk,dk,dv", [(1300, 1, 1, 200, 24), (1100, 2, 1, 256, 130), (1027, 3, 3, 129, 1), (1500, 1, 1, 2, 255)])
def test_wide_heads_in_segments(L, H, Hk, dk, dv, dtype):
    x, g, b, s0, do, ds = make(1, L, H, Hk, dk, dv, TYPES[dtype], seed=L)
    fwd, back = TOL[dtype]
    check_forward(x, g, b, s0, fwd)
    check_backward(x, g, b, s0, do, ds, back)


@pytest.mark.parametrize("dtype", TYPES)
def test_state_in_place_and_padded_rows_in_segments(dtype):
    x, g, b, s0, _, _ = make(2, 1200, 2, 2, 64, 96, TYPES[dtype], seed=33)
    o, s = api.delta_forward(*x, g, b, s0)
    here = s0.clone()
    o2, s2 = api.delta_forward(*x, g, b, here, out_state=here)
    assert s2 is here and torch.equal(o2, o) and torch.equal(here, s)
    g[1, 500:], b[1, 500:] = 0.0, 0.0   # the second row ends at 500
    _, s = check_forward(x, g, b, s0, TOL[dtype][0])
    _, short = api.delta_forward(*(t[1:, :500] for t in x), g[1:, :500], b[1:, :500], s0[1:])
    assert rel(s[1:], short.double().cpu()) <= F32_TOL


@pytest.mark.parametrize("dtype", TYPES)
def test_many_short_rows(dtype):
    fwd, back = TOL[dtype]
    for L in (1, 2, 33):
        x, g, b, s0, do, ds = make(150, L, 3, 1, 24, 40, TYPES[dtype], seed=34 + L)
        check_forward(x, g, b, s0, fwd)
        check_backward(x, g, b, s0, do, ds, back)


@pytest.mark.parametrize("dtype", TYPES)
def test_one_tensor_as_queries_keys_and_values(dtype):
    """The same memory three times, and rows that every batch row shares."""
    T = TYPES[dtype]
    fwd, back = TOL[dtype]
    x, g, b, _, do, _ = make(1, 90, 2, 2, 32, 32, T, seed=36)
    k = x[1].expand(3, 90, 2, 32)
    g, b = g.expand(3, 90, 2), b.expand(3, 90, 2)
    do = do.expand(3, 90, 2, 32)
    check_forward([k, k, k], g, b, None, fwd)
    check_backward([k, k, k], g, b, None, do, None, back)


def test_offsets_past_32_bits():
    """Batch rows 2^31 and more elements apart; states of more than 2^31 elements together."""
    far = (1 << 31) + 4096
    buf = torch.empty(far + (1 << 20), dtype=torch.bfloat16, device=DEV)
    x, g, b, s0, do, ds = make(2, 70, 2, 2, 64, 64, torch.bfloat16, seed=37)
    wide = []
    for n, t in enumerate((*x, do)):
        w = buf[n * (1 << 16):].as_strided(t.shape, (far, *t.stride()[1:]))
        w.copy_(t)
        wide.append(w)
    for a, c in zip(api.delta_forward(*wide[:3], g, b, s0), api.delta_forward(*x, g, b, s0)):
        assert torch.equal(a, c)
    for a, c in zip(api.delta_backward(*wide[:3], g, b, wide[3], s0, ds), api.delta_backward(*x, g, b, do, s0, ds)):
        assert torch.equal(a, c)
    w = torch.ones(64, device=DEV)
    for a, c in zip(api.headnorm_forward(wide[0], wide[1], w, w), api.headnorm_forward(x[0], x[1], w, w)):
        assert torch.equal(a, c)
    del buf, wide, w
    B, H, d = 1032, 128, 128
    state = torch.empty(B, H, d, d, device=DEV).fill_(0.25)
    q, k, v = (torch.randn(B, H, d, device=DEV) * d ** -0.5 for _ in range(3))
    g, b = torch.full((B, H), -0.1, device=DEV), torch.full((B, H), 0.5, device=DEV)
    want = api.delta_step(*(t[-2:].contiguous() for t in (q, k, v, g, b)), state[-2:].clone())
    o, _ = api.delta_step(q, k, v, g, b, state, out_state=state)
    assert torch.equal(o[-2:], want[0]) and torch.equal(state[-2:], want[1])


def test_two_streams_at_once():
    sets = [make(1, 900 + 50 * i, 2, 2, 64, 64, torch.bfloat16, seed=40 + i) for i in range(2)]

    def run(s):
        x, g, b, s0, do, ds = s
        w = torch.ones(64, device=DEV)
        return [*api.delta_forward(*x, g, b, s0), *api.delta_backward(*x, g, b, do, s0, ds),
                *api.headnorm_backward(x[0], x[1], g.abs() + 1, g.abs() + 1, x[0], x[1], w, w)]

    want = [run(s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(6):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                got[i].append(run(sets[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for out in got[i]:
            for a, c in zip(out, want[i]):
                assert torch.equal(a, c)


def test_long_gradients_in_bf16():
    check_backward(*make(2, 2500, 2, 1, 64, 64, torch.bfloat16, seed=42), 4e-3)


def test_head_norm_of_expanded_gradients_and_one_row():
    """A sum's gradient is one number for all elements; the same tensor as q and k."""
    q = torch.randn(2, 9, 4, 64, device=DEV, requires_grad=True)
    w = torch.randn(64, device=DEV, requires_grad=True)
    tab = sequence.rotary_table(9, 32, device=DEV)
    yq, yk = sequence.head_norm(q, q, w, w, tab)
    assert torch.equal(yq, yk)
    (yq.sum() + 2.0 * yk.sum()).backward()
    qd, wd = (t.detach().cpu().double().requires_grad_(True) for t in (q, w))
    pos = torch.arange(9).expand(2, 9)
    (3.0 * ref.headnorm(qd, wd, tab.cpu().double(), pos)[0].sum()).backward()
    assert rel(q.grad, qd.grad) <= 1e-6 and rel(w.grad, wd.grad) <= 1e-6
    y, none = sequence.head_norm(q.detach()[:1, :1], None, w.detach(), None, tab)
    assert none is None and torch.equal(y, yq.detach()[:1, :1])
