"""The trainable modules around the recurrences on the GPU: gradients against
torch's autograd through the fp64 formulas, capture in a HIP graph, and the
example model (training, prompt and single-token decoding).

Tolerances as for the kernels (fp32: 4e-6 of the 2-norm); a module adds a
library product on either side, whose fp32 rounding over 64 to 256 terms is
held to another 4e-6 each."""
import importlib.util
import os

import pytest
import torch

from nonlinear_rnn_solve_pararnn_amd import api, sequence
from tests import lm_ref
from tests.gpu_helpers import DEV, say

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def example():
    spec = importlib.util.spec_from_file_location("recurrent_lm", os.path.join(ROOT, "examples", "recurrent_lm.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def test_linear_attention_module():
    torch.manual_seed(0)
    m = sequence.LinearAttention(64, 4, 16, 24, device=DEV)
    x = torch.randn(2, 50, 64, device=DEV, requires_grad=True)
    s0 = torch.randn(2, 4, 16, 24, device=DEV, requires_grad=True)
    gy, gs = torch.randn(2, 50, 64, device=DEV), torch.randn(2, 4, 16, 24, device=DEV)
    y, s = m(x, s0)
    got = torch.autograd.grad((y * gy).sum() + (s * gs).sum(), [x, s0, m.qkv, m.out])
    xd, sd, wq, wo, gyd, gsd, g = (t.detach().cpu().double().requires_grad_(i < 4)
                                   for i, t in enumerate((x, s0, m.qkv, m.out, gy, gs, m.log_decay)))
    q, k, v = (t.unflatten(-1, (4, -1)) for t in (xd @ wq.T).split([64, 64, 96], -1))
    o, ref_s = lm_ref.linattn(q, k, v, g.detach(), sd)
    ref_y = o.flatten(2) @ wo.T
    want = torch.autograd.grad((ref_y * gyd).sum() + (ref_s * gsd).sum(), [xd, sd, wq, wo])
    errs = [lm_ref.rel(a, b.detach()) for a, b in zip((y, s, *got), (ref_y, ref_s, *want))]
    say("linear attention module", errs)
    assert max(errs) <= 3 * 4e-6, errs
    # a prompt, then single tokens
    with torch.no_grad():
        rows, st = [], m(x[:, :47])[1]
        for t in range(47, 50):
            o, st = m.step(x[:, t], st)
            rows.append(o)
        whole, fin = m(x)
    assert lm_ref.rel(torch.stack(rows, 1), whole[:, 47:].cpu().double()) <= 2 * 4e-6
    assert lm_ref.rel(st, fin.cpu().double()) <= 2 * 4e-6


def test_norm_and_embedding_modules():
    torch.manual_seed(1)
    emb = sequence.Embedding(100, 64, scale=8.0, padding_idx=7, device=DEV)
    norm = sequence.LayerNorm(64, device=DEV)
    with torch.no_grad():
        norm.weight.normal_(1.0, 0.1)
        norm.bias.normal_(0.0, 0.1)
    ids = torch.randint(0, 100, (3, 40), device=DEV)
    r = torch.randn(3, 40, 64, device=DEV, requires_grad=True)
    gy, gs = torch.randn(3, 40, 64, device=DEV), torch.randn(3, 40, 64, device=DEV)
    y, s = norm(emb(ids), r)
    got = torch.autograd.grad((y * gy).sum() + (s * gs).sum(), [emb.weight, norm.weight, norm.bias, r])
    ew, w, b, rd = (t.detach().cpu().double().requires_grad_(True) for t in (emb.weight, norm.weight, norm.bias, r))
    sd = ew[ids.cpu()] * 8.0 + rd
    yd, _, _ = lm_ref.layernorm(sd, w, b)
    want = list(torch.autograd.grad((yd * gy.cpu()).sum() + (sd * gs.cpu()).sum(), [ew, w, b, rd]))
    want[0][7] = 0
    errs = [lm_ref.rel(a, c.detach()) for a, c in zip((y, s, *got), (yd, sd, *want))]
    say("norm and embedding", errs)
    assert max(errs) <= 4e-6, errs


def test_bf16_module_and_expanded_gradient():
    """sum() hands the backward pass an expanded scalar."""
    m = sequence.LinearAttention(64, 2, 32, device=DEV, dtype=torch.bfloat16)
    x = torch.randn(2, 70, 64, device=DEV, dtype=torch.bfloat16, requires_grad=True)
    y, s = m(x)
    assert y.dtype == torch.bfloat16 and s.dtype == torch.float32
    q, k, v = (t.detach().requires_grad_(True) for t in m._project(x))
    o, _ = sequence.linear_attention(q, k, v, m.log_decay)
    o.sum().backward()
    ref = lm_ref.linattn_grads(*lm_ref.f64(q, k, v, m.log_decay), torch.ones(2, 70, 2, 32, dtype=torch.float64))
    for a, b in zip((q.grad, k.grad, v.grad), ref):
        assert lm_ref.rel(a, b) <= 4e-3


def test_graph_replays():
    """Every new operator captured in one HIP graph, replayed with inputs
    changed in place and eager calls between, each replay against eager."""
    gen = torch.Generator().manual_seed(2)
    r = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    ws = api.new_workspace(64 << 20, DEV)
    ids = torch.zeros(3000, dtype=torch.int64, device=DEV)
    table, grad = r(500, 64).to(DEV), r(3000, 64).to(DEV)
    w, b, g = r(64).to(DEV), r(64).to(DEV), -torch.rand(2, generator=gen).to(DEV)
    q, k, v, s0 = (t.to(DEV) for t in (r(1, 1500, 2, 32), r(1, 1500, 2, 32), r(1, 1500, 2, 32), r(1, 2, 32, 32)))

    def run():
        e = api.embedding_forward(ids, table, scale=2.0)
        y, s, mean, rstd = api.layernorm_forward(e, w, b, grad)
        lb = api.layernorm_backward(s, w, mean, rstd, grad, ws=ws)
        eb = api.embedding_backward(ids, grad, 500, ws=ws)
        o, st = api.linattn_forward(q, k, v, g, s0, ws=ws)
        gr = api.linattn_backward(q, k, v, g, o, s0, st, ws=ws)
        return [e, y, s, *lb, eb, o, st, *gr, *api.linattn_step(q[:, 0], k[:, 0], v[:, 0], g, st)]

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
        ids.copy_(torch.randint(0, 500, (3000,), generator=gen))
        for t in (grad, q, v):
            t.copy_(torch.randn(t.shape, generator=gen))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        for a, c in zip(got, run()):
            assert torch.equal(a, c), i
        torch.cuda.synchronize()


def test_example_model_learns_and_decodes():
    ex = example()
    torch.manual_seed(3)
    vocab = 64
    model = ex.RecurrentLM(vocab, dim=64, depth=2, heads=2, device=DEV)
    losses = ex.train(model, vocab, steps=40, B=8, L=100)
    say("losses", losses[0], losses[-1])
    # from log 64 = 4.2 (random) towards the text's own entropy, about 0.4
    assert losses[-1] < 0.5 * losses[0]
    ids = ex.text(2, 60, vocab, torch.Generator(device=DEV).manual_seed(4), DEV)
    with torch.no_grad():
        logits, _ = model(ids)
        _, states = model(ids[:, :50])
        states = [(h.contiguous(), s) for h, s in states]
        for t in range(50, 60):
            step, states = model.step(ids[:, t], states)
            # the prompt's Newton solve stops within 1e-4 of the recurrence that the steps follow
            assert float((step - logits[:, t]).abs().max()) <= 1e-2 * float(logits.abs().max())
    out = model.generate(ids, 5)
    assert out.shape == (2, 5) and bool(((out >= 0) & (out < vocab)).all())
