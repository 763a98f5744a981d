"""The delta-rule mixer's modules on the GPU: gradients against torch's autograd
through the fp64 formulas, prompts and single tokens, capture in a HIP graph,
and the example model with it.

Tolerances as for the kernels (fp32: 1.6e-5 of the 2-norm behind two
recurrences); a module adds library products and elementwise steps in fp32 on
either side, held to another 1.6e-5."""
import pytest
import torch

from nonlinear_rnn_solve_pararnn_amd import api, sequence
from tests import lm_ref, mixer_ref as ref
from tests.gpu_helpers import DEV, say
from tests.test_gpu_sequence import example

pytestmark = pytest.mark.gpu

TOL = 2 * 1.6e-5


def test_gated_delta_module():
    torch.manual_seed(0)
    m = sequence.GatedDelta(64, 4, 16, 24, key_heads=2, device=DEV)
    x = torch.randn(2, 50, 64, device=DEV, requires_grad=True)
    s0 = torch.randn(2, 4, 16, 24, device=DEV, requires_grad=True)
    gy, gs = torch.randn(2, 50, 64, device=DEV), torch.randn(2, 4, 16, 24, device=DEV)
    params = [m.qkv, m.gates, m.out, m.a, m.bias, m.norm]
    y, s = m(x, s0)
    got = torch.autograd.grad((y * gy).sum() + (s * gs).sum(), [x, s0, *params])
    xd, sd, qkv, gates, out, a, bias, norm = (t.detach().cpu().double().requires_grad_(True) for t in (x, s0, *params))
    q, k, v = (xd @ qkv.T).split([32, 32, 96], -1)
    q, k = (t.unflatten(-1, (2, 16)) for t in (q, k))
    q, k = (t * ((t * t).sum(-1, keepdim=True) + 1e-6) ** -0.5 for t in (q, k))
    z = xd @ gates.T
    o, rs = ref.delta(q, k, v.unflatten(-1, (4, 24)), -torch.exp(a) * torch.log1p(torch.exp(z[..., 4:] + bias)),
                      torch.sigmoid(z[..., :4]), sd)
    o = o * ((o * o).sum(-1, keepdim=True) / 24 + 1e-6) ** -0.5 * norm
    ry = o.flatten(2) @ out.T
    want = torch.autograd.grad((ry * gy.cpu().double()).sum() + (rs * gs.cpu().double()).sum(), [xd, sd, qkv, gates, out, a, bias, norm])
    errs = [lm_ref.rel(p, w.detach()) for p, w in zip((y, s, *got), (ry, rs, *want))]
    say("gated delta module", errs)
    assert max(errs) <= TOL, errs
    with torch.no_grad():  # a prompt, then single tokens
        rows, st = [], m(x[:, :47])[1]
        for t in range(47, 50):
            r, st = m.step(x[:, t], st)
            rows.append(r)
        whole, fin = m(x)
    assert lm_ref.rel(torch.stack(rows, 1), whole[:, 47:].cpu().double()) <= TOL
    assert lm_ref.rel(st, fin.cpu().double()) <= TOL


def test_linear_attention_with_norms_and_rotation():
    torch.manual_seed(1)
    m = sequence.LinearAttention(64, 4, 16, 24, norm="rms", rotary=8, max_positions=200, device=DEV)
    with torch.no_grad():
        m.q_weight.normal_(1.0, 0.1)
        m.k_weight.normal_(1.0, 0.1)
    x = torch.randn(2, 40, 64, device=DEV, requires_grad=True)
    gy = torch.randn(2, 40, 64, device=DEV)
    pos = (torch.tensor([[3], [150]]) + torch.arange(40)).to(DEV)
    y, s = m(x, None, pos)
    params = [m.qkv, m.out, m.q_weight, m.k_weight]
    got = torch.autograd.grad((y * gy).sum(), [x, *params])
    xd, qkv, out, wq, wk = (t.detach().cpu().double().requires_grad_(True) for t in (x, *params))
    q, k, v = (t.unflatten(-1, (4, -1)) for t in (xd @ qkv.T).split([64, 64, 96], -1))
    tab = m.table.cpu().double()
    q, k = ref.headnorm(q, wq, tab, pos.cpu())[0], ref.headnorm(k, wk, tab, pos.cpu())[0]
    o, _ = lm_ref.linattn(q, k, v, m.log_decay.cpu().double())
    want = torch.autograd.grad(((o.flatten(2) @ out.T) * gy.cpu().double()).sum(), [xd, qkv, out, wq, wk])
    errs = [lm_ref.rel(a, b.detach()) for a, b in zip((y, *got), (o.flatten(2) @ out.T, *want))]
    say("normed linear attention", errs)
    assert max(errs) <= TOL, errs
    with torch.no_grad():
        st = m(x[:, :39], None, pos[:, :39].contiguous())[1]
        r, st = m.step(x[:, 39], st, pos[:, 39].contiguous())
    assert lm_ref.rel(r, y[:, 39].detach().cpu().double()) <= TOL
    assert torch.equal(m(x)[0], m(x, None, torch.arange(40, device=DEV).expand(2, 40).contiguous())[0])


def test_bf16_module_and_expanded_gradient():
    m = sequence.GatedDelta(64, 2, 32, device=DEV, dtype=torch.bfloat16)
    x = torch.randn(2, 70, 64, device=DEV, dtype=torch.bfloat16, requires_grad=True)
    y, s = m(x)
    assert y.dtype == torch.bfloat16 and s.dtype == torch.float32
    ops = [t.detach().requires_grad_(True) for t in m._operands(x)]
    o, _ = sequence.gated_delta(*ops)
    o.sum().backward()
    want = ref.delta_grads(*lm_ref.f64(*ops), torch.ones(2, 70, 2, 32, dtype=torch.float64))
    for n, (a, b) in enumerate(zip(ops, want)):
        assert lm_ref.rel(a.grad, b) <= (4e-3 if n < 3 else 1.6e-5)
    y.sum().backward()
    assert all(bool(torch.isfinite(p.grad).all()) for p in m.parameters())


def test_graph_replays():
    """All of the mixer's operators in one HIP graph, with segments, shared heads and weight gradients, replayed with
    inputs changed in place and eager calls between, each replay against eager."""
    gen = torch.Generator().manual_seed(2)
    r = lambda *s: torch.randn(*s, generator=gen).to(DEV)  # noqa: E731
    q, k, v, s0 = r(1, 1500, 2, 64), r(1, 1500, 2, 64), r(1, 1500, 4, 32), r(1, 4, 64, 32)
    g, b, w, tab = -torch.rand(1, 1500, 4, generator=gen).to(DEV), torch.rand(1, 1500, 4, generator=gen).to(DEV), r(64), sequence.rotary_table(1500, 32, device=DEV)

    def run():
        yq, yk, rq, rk = api.headnorm_forward(q, k, w, w, tab, kind="l2")
        o, st = api.delta_forward(yq, yk, v, g, b, s0)
        grads = api.delta_backward(yq, yk, v, g, b, o, s0, st)
        hb = api.headnorm_backward(q, k, rq, rk, grads[0], grads[1], w, w, tab, kind="l2")
        return [yq, yk, o, st, *grads, *hb, *api.delta_step(yq[:, 0], yk[:, 0], v[:, 0], g[:, 0], b[:, 0], st)]

    run()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    for i in range(4):
        for t in (q, k, v):
            t.copy_(torch.randn(t.shape, generator=gen))
        b.copy_(torch.rand(b.shape, generator=gen))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        for n, (a, c) in enumerate(zip(got, run())):
            assert torch.equal(a, c), (i, n)
        torch.cuda.synchronize()


def test_two_graphs_and_eager_calls_share_nothing():
    """Two captured graphs and eager calls in between: each keeps a workspace of its own."""
    gen = torch.Generator().manual_seed(5)
    sets = []
    for L in (900, 300):
        q, k = (torch.randn(1, L, 2, 32, generator=gen).to(DEV) * 32 ** -0.5 for _ in range(2))
        v, do = (torch.randn(1, L, 2, 48, generator=gen).to(DEV) for _ in range(2))
        g, b = -torch.rand(1, L, 2, generator=gen).to(DEV), torch.rand(1, L, 2, generator=gen).to(DEV)
        sets.append((q, k, v, g, b, do))
    run = lambda q, k, v, g, b, do: [*api.delta_forward(q, k, v, g, b), *api.delta_backward(q, k, v, g, b, do)[:5]]  # noqa: E731
    want = [[t.clone() for t in run(*s)] for s in sets]
    torch.cuda.synchronize()
    graphs = []
    for s in sets:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = run(*s)
        graphs.append((graph, out))
    for i in (0, 1, 1, 0, 1):
        graphs[i][0].replay()
        run(*sets[1 - i])
        torch.cuda.synchronize()
        for a, c in zip(graphs[i][1], want[i]):
            assert torch.equal(a, c)


def test_example_model_with_the_delta_rule():
    ex = example()
    torch.manual_seed(3)
    vocab = 64
    model = ex.RecurrentLM(vocab, dim=64, depth=2, heads=2, device=DEV, mixer="delta")
    losses = ex.train(model, vocab, steps=3, B=4, L=100)
    assert all(x == x and x < float("inf") for x in losses)
    assert all(p.grad is not None and bool(torch.isfinite(p.grad).all()) for p in model.parameters())
    ids = ex.text(2, 60, vocab, torch.Generator(device=DEV).manual_seed(4), DEV)
    with torch.no_grad():
        logits, _ = model(ids)
        _, states = model(ids[:, :50])
        states = [(h.contiguous(), s) for h, s in states]
        for t in range(50, 60):
            step, states = model.step(ids[:, t], states)
            # the prompt's Newton solve stops within 1e-4 of the recurrence that the steps follow
            assert float((step - logits[:, t]).abs().max()) <= 1e-2 * float(logits.abs().max())
    assert model.generate(ids, 5).shape == (2, 5)
