"""A small recurrent language model on the framework's kernels: embedding, then
blocks of [layer norm, ParaGRU, residual] and [layer norm, a mixer with a matrix
state, residual], a last norm and tied output weights.  The mixer is linear
attention or the gated delta rule.

    python examples/recurrent_lm.py [--mixer delta]

trains it for some steps on synthetic text (a fixed random walk over tokens,
which the model can learn) and decodes a continuation: the prompt in one
pass, then token by token with the carried states.  Needs an MI355X.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch
import torch.nn.functional as F

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from nonlinear_rnn_solve_pararnn_amd import api, layers, sequence  # noqa: E402


class Block(torch.nn.Module):
    def __init__(self, dim, heads, device, mixer="linear"):
        super().__init__()
        self.norm1, self.norm2 = (sequence.LayerNorm(dim, device=device) for _ in range(2))
        self.gru = layers.ParaGRU(dim, dim, device=device)
        kind = {"linear": sequence.LinearAttention, "delta": sequence.GatedDelta}[mixer]
        self.attention = kind(dim, heads, dim // heads, device=device)

    def forward(self, x, residual, state=None):
        """x is what the sublayer before computed, residual the stream it joins; returns the same pair and the states."""
        h0, s = (None, None) if state is None else state
        y, stream = self.norm1(x, residual) if residual is not None else (self.norm1(x), x)
        y = self.gru(y, h0)
        h = y[:, -1]
        y, stream = self.norm2(y, stream)
        y, s = self.attention(y, s)
        return y, stream, (h, s)

    @torch.no_grad()
    def step(self, x, residual, state):
        """One token: x, residual [B, D]."""
        h, s = state
        y, stream = self.norm1(x, residual) if residual is not None else (self.norm1(x), x)
        p = self.gru.project(y[:, None])
        h = api.gru_sequential(*p, *self.gru.u, h)[:, 0]
        y, stream = self.norm2(h.contiguous(), stream)
        y, s = self.attention.step(y, s)
        return y, stream, (h.contiguous(), s)


class RecurrentLM(torch.nn.Module):
    def __init__(self, vocab, dim=256, depth=2, heads=4, device="cuda", mixer="linear"):
        super().__init__()
        self.embedding = sequence.Embedding(vocab, dim, scale=dim ** 0.5, device=device)
        self.blocks = torch.nn.ModuleList(Block(dim, heads, device, mixer) for _ in range(depth))
        self.norm = sequence.LayerNorm(dim, device=device)

    def forward(self, ids, states=None):
        """Logits [B, L, V] of ids [B, L], and the states after the last token."""
        x, stream, out = self.embedding(ids), None, []
        for i, block in enumerate(self.blocks):
            x, stream, state = block(x, stream, None if states is None else states[i])
            out.append(state)
        y, _ = self.norm(x, stream)
        return F.linear(y, self.embedding.weight), out

    @torch.no_grad()
    def step(self, ids, states):
        """Logits [B, V] of one token each, ids [B]."""
        x, stream, out = self.embedding(ids), None, []
        for block, state in zip(self.blocks, states):
            x, stream, state = block.step(x, stream, state)
            out.append(state)
        y, _ = self.norm(x, stream)
        return F.linear(y, self.embedding.weight), out

    @torch.no_grad()
    def generate(self, prompt, count):
        """The `count` most likely next tokens after prompt [B, L], one after the other."""
        logits, states = self(prompt)
        states = [(h.contiguous(), s) for h, s in states]
        tokens = [logits[:, -1].argmax(-1)]
        for _ in range(count - 1):
            logits, states = self.step(tokens[-1], states)
            tokens.append(logits.argmax(-1))
        return torch.stack(tokens, 1)


def text(B, L, vocab, generator, device):
    """Walks over tokens: each goes to one of two fixed successors, the first nine times in ten."""
    table = torch.randint(0, vocab, (vocab, 2), generator=torch.Generator().manual_seed(1)).to(device)
    ids = torch.randint(0, vocab, (B,), generator=generator, device=device)
    rare = (torch.rand(B, L, generator=generator, device=device) < 0.1).long()
    out = []
    for t in range(L):
        out.append(ids)
        ids = table[ids, rare[:, t]]
    return torch.stack(out, 1)


def train(model, vocab, steps, B, L, lr=3e-3, seed=0, report=None):
    device = model.norm.weight.device
    gen = torch.Generator(device=device).manual_seed(seed)
    opt = torch.optim.AdamW(model.parameters(), lr=lr)
    losses = []
    for i in range(steps):
        ids = text(B, L + 1, vocab, gen, device)
        logits, _ = model(ids[:, :-1])
        loss = F.cross_entropy(logits.flatten(0, 1), ids[:, 1:].flatten())
        opt.zero_grad(set_to_none=True)
        loss.backward()
        opt.step()
        losses.append(loss.detach())
        if report is not None:
            report(i, losses[-1])
    return [float(x) for x in losses]


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--vocab", type=int, default=512)
    ap.add_argument("--dim", type=int, default=256)
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--batch", type=int, default=16)
    ap.add_argument("--length", type=int, default=512)
    ap.add_argument("--mixer", choices=("linear", "delta"), default="linear")
    a = ap.parse_args()
    torch.manual_seed(0)
    model = RecurrentLM(a.vocab, a.dim, mixer=a.mixer)
    train(model, a.vocab, a.steps, a.batch, a.length,
          report=lambda i, x: print("step %d loss %.3f" % (i, float(x)), flush=True) if i % 10 == 0 or i == a.steps - 1 else None)
    prompt = text(2, 64, a.vocab, torch.Generator(device="cuda").manual_seed(9), "cuda")
    print("continuations:", model.generate(prompt, 16).tolist())


if __name__ == "__main__":
    main()
