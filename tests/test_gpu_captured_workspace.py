"""Calls without a workspace of their own, captured in a HIP graph: replays
depend on no buffer that later calls on the stream grow, replace or use."""
import pytest
import torch

from nonlinear_rnn_solve_pararnn_amd import api, sequence
from tests.gpu_helpers import DEV

pytestmark = pytest.mark.gpu


def test_captured_modules_after_larger_calls():
    torch.manual_seed(0)
    V, D, B, L = 600, 64, 2, 1500
    emb = sequence.Embedding(V, D, scale=8.0, device=DEV)
    norm = sequence.LayerNorm(D, device=DEV)
    mix = sequence.LinearAttention(D, 2, 32, device=DEV)
    params = [*emb.parameters(), *norm.parameters(), *mix.parameters()]
    gen = torch.Generator().manual_seed(1)
    ids = torch.randint(0, V, (B, L), generator=gen).to(DEV)
    weight = torch.randn(B, L, D, generator=gen).to(DEV)
    a, b = torch.rand(B, L, D, generator=gen).to(DEV), torch.randn(B, L, D, generator=gen).to(DEV)

    def run(ids=ids, weight=weight, a=a, b=b):
        x = emb(ids)
        y, s = mix(norm(x))
        grads = torch.autograd.grad((y * weight).mean() + s.mean(), params)
        return [y.detach(), s.detach(), *grads, api.linscan_diag(a, b)]

    def larger():
        n = 9
        run(ids.repeat(n, 2), weight.repeat(n, 2, 1), a.repeat(n, 2, 1), b.repeat(n, 2, 1))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
        run()
    torch.cuda.synchronize()
    kept = {id(x) for d in api._all_kept for x in d.values()}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out = run()
    assert {id(x) for d in api._all_kept for x in d.values()} == kept
    with torch.cuda.stream(side):
        larger()
    torch.cuda.synchronize()
    for i in range(4):
        ids.copy_(torch.randint(0, V, (B, L), generator=gen))
        weight.copy_(torch.randn(B, L, D, generator=gen))
        a.copy_(torch.rand(B, L, D, generator=gen))
        # memory that the calls have let go of, written over by others
        fill = [torch.full((1 << 22,), 0xff, dtype=torch.uint8, device=DEV) for _ in range(16)]
        with torch.cuda.stream(side):
            fill += [torch.full((1 << 22,), 0xff, dtype=torch.uint8, device=DEV) for _ in range(16)]
            graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        assert all(bool((t == 0xff).all()) for t in fill), i  # and the replay wrote over none of it
        del fill
        for p, q in zip(got, run()):
            assert torch.equal(p, q), i
        with torch.cuda.stream(side):
            larger()
        torch.cuda.synchronize()


def test_two_graphs_of_one_stream_side_by_side():
    """Captured one after the other on one stream, replayed on two."""
    gen = torch.Generator().manual_seed(2)
    sets = []
    for i in range(2):
        q, k, v = (torch.randn(1, 4000, 2, 64, generator=gen).to(DEV) for _ in range(3))
        sets.append((q, k, v, -0.1 * torch.rand(2, generator=gen).to(DEV)))
    want = [api.linattn_forward(*s) for s in sets]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        api.linattn_forward(*sets[0])
    torch.cuda.synchronize()
    graphs, outs = [], []
    for s in sets:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            outs.append(api.linattn_forward(*s))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert torch.equal(o[0], w[0]) and torch.equal(o[1], w[1])
