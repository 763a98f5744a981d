"""What a sequence model has around the recurrences, trainable: the embedding
lookup, layer norm with the residual sum before it, linear attention with a
decay per head, the gated delta rule, and norms of queries and keys for each
head with the position rotation, on the kernels of libpararnn.so (forward and
gradients).

``Embedding`` turns tokens into x [B, L, D], ``LayerNorm`` stands before each
mixing layer (``ParaGRU`` / ``ParaLSTM`` of layers.py, or ``LinearAttention``
or ``GatedDelta`` here), and takes the residual sum along, so the sum is
written and normed in one pass.  ``LinearAttention`` and ``GatedDelta`` carry a
[dk, dv] state per head from call to call: whole prompts through ``forward``,
single tokens through ``step``.

Activations are fp32 or bf16; norm weights, decays and states are fp32.  There
is no CPU path: the kernels raise unless their inputs are on a HIP device.
"""
from __future__ import annotations

import math
from typing import Optional

import torch
import torch.nn.functional as F
from torch.autograd.function import once_differentiable

from . import api


def _rows_dense(t: Optional[torch.Tensor]):
    """t with a dense last dimension (gradients may come as expanded scalars)."""
    return t if t is None or t.shape[-1] == 1 or t.stride(-1) == 1 else t.contiguous()


class LinattnFunction(torch.autograd.Function):
    """(o, final state) of api.linattn_forward, with its gradients for q, k, v
    and the initial state.  The log decay is a constant."""

    @staticmethod
    def forward(ctx, q, k, v, log_decay, state, scale):
        if ctx.needs_input_grad[3]:
            raise ValueError("log_decay is a constant of linear attention and has no gradient")
        o, out_state = api.linattn_forward(q, k, v, log_decay, state, scale=scale)
        ctx.save_for_backward(q, k, v, log_decay, state)
        ctx.scale = scale
        ctx.set_materialize_grads(False)
        return o, out_state

    @staticmethod
    @once_differentiable
    def backward(ctx, go, gstate):
        q, k, v, log_decay, state = ctx.saved_tensors
        if go is None and gstate is None:
            return (None,) * 6
        if go is None:
            go = torch.zeros_like(v, memory_format=torch.contiguous_format)
        gstate = None if gstate is None else gstate.contiguous()
        gq, gk, gv, gs = api.linattn_backward(q, k, v, log_decay, _rows_dense(go), state, gstate, scale=ctx.scale,
                                              want_state=state is not None and ctx.needs_input_grad[4])
        return gq, gk, gv, None, gs, None


class LayerNormFunction(torch.autograd.Function):
    """(y, s) of api.layernorm_forward: s = x + residual, y its norm."""

    @staticmethod
    def forward(ctx, x, weight, bias, residual, eps):
        y, s, mean, rstd = api.layernorm_forward(x, weight, bias, residual, eps=eps)
        ctx.save_for_backward(s, weight, mean, rstd)
        ctx.set_materialize_grads(False)
        if residual is None:
            s = s.view_as(s)  # x itself: an output of its own for autograd
        return y, s

    @staticmethod
    @once_differentiable
    def backward(ctx, gy, gs):
        s, weight, mean, rstd = ctx.saved_tensors
        need = ctx.needs_input_grad
        if gy is None:
            return gs, None, None, gs if need[3] else None, None
        gx, gw, gb = api.layernorm_backward(s, weight, mean, rstd, gy.contiguous(), None if gs is None else gs.contiguous(),
                                            want_w=need[1], want_b=need[2])
        return gx, gw, gb, gx if need[3] else None, None


class EmbeddingFunction(torch.autograd.Function):
    """scale * table[ids]; the table's gradient by sorted tokens."""

    @staticmethod
    def forward(ctx, ids, table, scale, padding_idx):
        ctx.save_for_backward(ids)
        ctx.rows, ctx.scale, ctx.padding_idx = table.shape[0], scale, padding_idx
        return api.embedding_forward(ids, table, scale=scale)

    @staticmethod
    @once_differentiable
    def backward(ctx, g):
        (ids,) = ctx.saved_tensors
        return None, api.embedding_backward(ids, g.contiguous(), ctx.rows, scale=ctx.scale,
                                            padding_idx=ctx.padding_idx), None, None


class DeltaFunction(torch.autograd.Function):
    """(o, final state) of api.delta_forward, with all of its gradients."""

    @staticmethod
    def forward(ctx, q, k, v, log_decay, beta, state, scale):
        o, out_state = api.delta_forward(q, k, v, log_decay, beta, state, scale=scale)
        ctx.save_for_backward(q, k, v, log_decay, beta, state)
        ctx.scale = scale
        ctx.set_materialize_grads(False)
        return o, out_state

    @staticmethod
    @once_differentiable
    def backward(ctx, go, gstate):
        q, k, v, log_decay, beta, state = ctx.saved_tensors
        if go is None and gstate is None:
            return (None,) * 7
        if go is None:
            go = torch.zeros_like(v, memory_format=torch.contiguous_format)
        gstate = None if gstate is None else gstate.contiguous()
        out = api.delta_backward(q, k, v, log_decay, beta, _rows_dense(go), state, gstate, scale=ctx.scale,
                                 want_state=state is not None and ctx.needs_input_grad[5])
        return *out, None


class HeadNormFunction(torch.autograd.Function):
    """Outputs of api.headnorm_forward: of q and k, or of q alone (and None)."""

    @staticmethod
    def forward(ctx, q, k, q_weight, k_weight, table, positions, kind, eps, interleaved):
        yq, yk, rq, rk = api.headnorm_forward(q, k, q_weight, k_weight, table, positions, kind=kind, eps=eps,
                                              interleaved=interleaved)
        ctx.save_for_backward(q, k, rq, rk, q_weight, k_weight, table, positions)
        ctx.kind, ctx.interleaved = kind, interleaved
        ctx.set_materialize_grads(False)
        return yq, yk

    @staticmethod
    @once_differentiable
    def backward(ctx, gq, gk):
        q, k, rq, rk, q_weight, k_weight, table, positions = ctx.saved_tensors
        if gq is None and gk is None:
            return (None,) * 9
        gq = torch.zeros_like(q, memory_format=torch.contiguous_format) if gq is None else _rows_dense(gq)
        if k is not None:
            gk = torch.zeros_like(k, memory_format=torch.contiguous_format) if gk is None else _rows_dense(gk)
        return *api.headnorm_backward(q, k, rq, rk, gq, gk, q_weight, k_weight, table, positions, kind=ctx.kind,
                                      interleaved=ctx.interleaved), None, None, None, None, None


def linear_attention(q, k, v, log_decay, state=None, *, scale=None):
    """Differentiable api.linattn_forward: (o, final state)."""
    return LinattnFunction.apply(q, k, v, log_decay, state, scale)


def gated_delta(q, k, v, log_decay, beta, state=None, *, scale=None):
    """Differentiable api.delta_forward: (o, final state)."""
    return DeltaFunction.apply(q, k, v, log_decay, beta, state, scale)


def head_norm(q, k=None, q_weight=None, k_weight=None, table=None, positions=None, *, kind="rms", eps=1e-6,
              interleaved=False):
    """Differentiable api.headnorm_forward: (yq, yk), yk None without k.  The
    table and the positions are constants."""
    return HeadNormFunction.apply(q, k, q_weight, k_weight, table, positions, kind, eps, interleaved)


def rotary_table(length: int, dim: int, *, base: float = 10000.0, device=None) -> torch.Tensor:
    """[length, dim] fp32 for head_norm: row t holds the cosines, then the
    sines, of the angles t base^(-2i / dim), worked out in 64 bits."""
    if length < 1 or dim < 2 or dim % 2:
        raise ValueError("length must be positive and dim even, got %d and %d" % (length, dim))
    rate = base ** (-torch.arange(0, dim, 2, dtype=torch.float64) / dim)
    angle = torch.arange(length, dtype=torch.float64)[:, None] * rate
    return torch.cat([angle.cos(), angle.sin()], 1).float().to(device)


def layer_norm(x, weight=None, bias=None, residual=None, *, eps=1e-5):
    """Differentiable api.layernorm_forward: (y, s), s = x + residual (x without
    one).  Operands that are not dense are copied."""
    return LayerNormFunction.apply(x.contiguous(), weight, bias, None if residual is None else residual.contiguous(), eps)


def embedding(ids, table, *, scale=1.0, padding_idx=None):
    """Differentiable api.embedding_forward.  Ids that are not dense are copied."""
    return EmbeddingFunction.apply(ids.contiguous(), table, scale, padding_idx)


class Embedding(torch.nn.Module):
    """Tokens [...] to rows [..., D], times `scale`; the gradient of row
    `padding_idx` is zero."""

    def __init__(self, num_rows: int, dim: int, *, scale: float = 1.0, padding_idx: Optional[int] = None, device=None,
                 dtype=torch.float32):
        super().__init__()
        if num_rows < 1 or dim < 1:
            raise ValueError("num_rows and dim must be positive")
        if padding_idx is not None and not 0 <= padding_idx < num_rows:
            raise ValueError("padding_idx must be in [0, %d), got %s" % (num_rows, padding_idx))
        self.scale, self.padding_idx = float(scale), padding_idx
        self.weight = torch.nn.Parameter(torch.empty(num_rows, dim, device=device, dtype=dtype))
        with torch.no_grad():
            self.weight.normal_(std=dim ** -0.5)

    def forward(self, ids: torch.Tensor) -> torch.Tensor:
        return embedding(ids, self.weight, scale=self.scale, padding_idx=self.padding_idx)

    def extra_repr(self):
        return "%d, %d, scale=%g, padding_idx=%s" % (*self.weight.shape, self.scale, self.padding_idx)


class LayerNorm(torch.nn.Module):
    """Layer norm of the last dimension.  forward(x) -> y;
    forward(x, residual) -> (y, s) with s = x + residual and y its norm."""

    def __init__(self, dim: int, *, eps: float = 1e-5, bias: bool = True, device=None):
        super().__init__()
        if dim < 1 or not eps >= 0.0:
            raise ValueError("dim must be positive and eps >= 0")
        self.eps = float(eps)
        self.weight = torch.nn.Parameter(torch.ones(dim, device=device, dtype=torch.float32))
        self.bias = torch.nn.Parameter(torch.zeros(dim, device=device, dtype=torch.float32)) if bias else None

    def forward(self, x: torch.Tensor, residual: Optional[torch.Tensor] = None):
        y, s = layer_norm(x, self.weight, self.bias, residual, eps=self.eps)
        return y if residual is None else (y, s)

    def extra_repr(self):
        return "%d, eps=%g, bias=%s" % (self.weight.numel(), self.eps, self.bias is not None)


class LinearAttention(torch.nn.Module):
    """Linear attention with a fixed decay per head, with its projections:

        q, k, v = x W^T (heads of dk, dk, dv),  S_t = e^g S_{t-1} + k_t^T v_t,
        o_t = dk^-1/2 q_t S_t,  y = o W_o^T.

    forward(x [B, L, D], state or None) -> (y [B, L, D], state [B, H, dk, dv]);
    step(x [B, D], state) -> (y [B, D], state), which it updates in place.
    `log_decay` [H] (a buffer) defaults to log(1 - 2^-n), n spread from 3 to 9:
    memories from some 8 to some 500 positions.

    norm="rms" (with weights) or "l2": q and k of each head are normed first,
    and their first `rotary` elements turned by their position, below
    `max_positions`.  forward and step then take positions ([B, L] and [B]);
    without them forward counts from 0."""

    def __init__(self, dim: int, heads: int, dk: int, dv: Optional[int] = None, *, log_decay: Optional[torch.Tensor] = None,
                 norm: Optional[str] = None, rotary: int = 0, max_positions: int = 2048, device=None, dtype=torch.float32):
        super().__init__()
        dv = dk if dv is None else dv
        if min(dim, heads, dk, dv) < 1 or max(dk, dv) > api.MAX_HEAD_DIM:
            raise ValueError("sizes must be positive and heads at most %d wide" % api.MAX_HEAD_DIM)
        if norm is not None and norm not in api.NORM_KINDS:
            raise ValueError("norm must be 'rms' or 'l2', got %r" % (norm,))
        if rotary < 0 or rotary % 2 or rotary > dk or (rotary and norm is None):
            raise ValueError("rotary must be even, at most dk and with a norm, got %d" % rotary)
        self.dim, self.heads, self.dk, self.dv = dim, heads, dk, dv
        self.norm = norm
        self.q_weight, self.k_weight = (torch.nn.Parameter(torch.ones(dk, device=device)) if norm == "rms" else None
                                        for _ in range(2))
        self.register_buffer("table", rotary_table(max_positions, rotary, device=device) if rotary else None, persistent=False)
        self.qkv = torch.nn.Parameter(torch.empty(heads * (2 * dk + dv), dim, device=device, dtype=dtype))
        self.out = torch.nn.Parameter(torch.empty(dim, heads * dv, device=device, dtype=dtype))
        if log_decay is None:
            log_decay = torch.log1p(-torch.exp2(-torch.linspace(3.0, 9.0, heads)))
        if log_decay.shape != (heads,) or log_decay.requires_grad:
            raise ValueError("log_decay must be a constant [heads] tensor")
        self.register_buffer("log_decay", log_decay.detach().to(device=device, dtype=torch.float32))
        with torch.no_grad():
            for w in (self.qkv, self.out):
                w.uniform_(-1.0 / math.sqrt(w.shape[1]), 1.0 / math.sqrt(w.shape[1]))

    def _project(self, x):
        """q, k, v as views of one product (the kernels take their strides)."""
        H, dk, dv = self.heads, self.dk, self.dv
        p = F.linear(x, self.qkv)
        q, k, v = p.split([H * dk, H * dk, H * dv], -1)
        return [t.unflatten(-1, (H, d)) for t, d in ((q, dk), (k, dk), (v, dv))]

    def _normed(self, q, k, v, positions):
        if self.norm is None:
            if positions is not None:
                raise ValueError("positions are given to a layer without rotation")
            return q, k, v
        q, k = head_norm(q, k, self.q_weight, self.k_weight, self.table, positions, kind=self.norm)
        return q, k, v

    def forward(self, x: torch.Tensor, state: Optional[torch.Tensor] = None, positions: Optional[torch.Tensor] = None):
        if x.dim() != 3 or x.shape[-1] != self.dim:
            raise ValueError("x must be [B, L, %d], got %s" % (self.dim, tuple(x.shape)))
        o, state = linear_attention(*self._normed(*self._project(x), positions), self.log_decay, state)
        return F.linear(o.flatten(2), self.out), state

    @torch.no_grad()
    def step(self, x: torch.Tensor, state: torch.Tensor, positions: Optional[torch.Tensor] = None):
        if x.dim() != 2 or x.shape[-1] != self.dim:
            raise ValueError("x must be [B, %d], got %s" % (self.dim, tuple(x.shape)))
        o, state = api.linattn_step(*self._normed(*self._project(x), positions), self.log_decay, state, out_state=state)
        if not state.is_inference():  # autograd learns of the change where the state was saved
            torch.autograd.graph.increment_version(state)
        return F.linear(o.flatten(1), self.out), state

    def extra_repr(self):
        return "%d, heads=%d, dk=%d, dv=%d" % (self.dim, self.heads, self.dk, self.dv)


class GatedDelta(torch.nn.Module):
    """The gated delta rule with its projections, gates and norms:

        q, k = x W^T (key_heads heads of dk), each of unit length,  v = x W^T (heads of dv),
        b = sigmoid(x W_b^T),  g = -exp(a) softplus(x W_g^T + bias),
        S_t = e^(g_t) (I - b_t k_t^T k_t) S_{t-1} + b_t k_t^T v_t,  o_t = dk^-1/2 q_t S_t,
        y = n(o) W_o^T,  n the RMS norm of each head with a weight.

    forward(x [B, L, D], state or None) -> (y [B, L, D], state [B, H, dk, dv]);
    step(x [B, D], state) -> (y [B, D], state), which it updates in place.
    The gates begin with decays of about a 2^-n part a position, n spread over
    the heads from 3 to 9."""

    def __init__(self, dim: int, heads: int, dk: int, dv: Optional[int] = None, *, key_heads: Optional[int] = None,
                 eps: float = 1e-6, device=None, dtype=torch.float32):
        super().__init__()
        dv = dk if dv is None else dv
        key_heads = heads if key_heads is None else key_heads
        if min(dim, heads, key_heads) < 1 or min(dk, dv) < 2 or max(dk, dv) > api.MAX_HEAD_DIM:
            raise ValueError("sizes must be positive, heads 2 to %d wide" % api.MAX_HEAD_DIM)
        if heads % key_heads:
            raise ValueError("heads must be a multiple of key_heads, got %d and %d" % (heads, key_heads))
        self.dim, self.heads, self.key_heads, self.dk, self.dv, self.eps = dim, heads, key_heads, dk, dv, float(eps)
        make = lambda *s, t=dtype: torch.nn.Parameter(torch.empty(*s, device=device, dtype=t))  # noqa: E731
        self.qkv = make(2 * key_heads * dk + heads * dv, dim)
        self.gates = make(2 * heads, dim)                       # beta's rows, then the decay's
        self.out = make(dim, heads * dv)
        self.a = make(heads, t=torch.float32)                   # log of the decay's rate
        self.bias = make(heads, t=torch.float32)
        self.norm = torch.nn.Parameter(torch.ones(dv, device=device, dtype=torch.float32))
        with torch.no_grad():
            for w in (self.qkv, self.gates, self.out):
                w.uniform_(-1.0 / math.sqrt(w.shape[1]), 1.0 / math.sqrt(w.shape[1]))
            # softplus of a bias of 0 is log 2
            self.a.copy_(-torch.linspace(3.0, 9.0, heads) * math.log(2.0) - math.log(math.log(2.0)))
            self.bias.zero_()

    def _operands(self, x):
        """q, k, v, the log decay and beta of the delta rule."""
        H, Hk, dk, dv = self.heads, self.key_heads, self.dk, self.dv
        q, k, v = F.linear(x, self.qkv).split([Hk * dk, Hk * dk, H * dv], -1)
        q, k = head_norm(q.unflatten(-1, (Hk, dk)), k.unflatten(-1, (Hk, dk)), kind="l2", eps=self.eps)
        b, g = F.linear(x, self.gates).float().split(H, -1)
        return q, k, v.unflatten(-1, (H, dv)), -torch.exp(self.a) * F.softplus(g + self.bias), torch.sigmoid(b)

    def _output(self, o):
        return F.linear(head_norm(o, None, self.norm, eps=self.eps)[0].flatten(-2), self.out)

    def forward(self, x: torch.Tensor, state: Optional[torch.Tensor] = None):
        if x.dim() != 3 or x.shape[-1] != self.dim:
            raise ValueError("x must be [B, L, %d], got %s" % (self.dim, tuple(x.shape)))
        o, state = gated_delta(*self._operands(x), state)
        return self._output(o), state

    @torch.no_grad()
    def step(self, x: torch.Tensor, state: torch.Tensor):
        if x.dim() != 2 or x.shape[-1] != self.dim:
            raise ValueError("x must be [B, %d], got %s" % (self.dim, tuple(x.shape)))
        o, state = api.delta_step(*self._operands(x), state, out_state=state)
        if not state.is_inference():  # autograd learns of the change where the state was saved
            torch.autograd.graph.increment_version(state)
        return self._output(o), state

    def extra_repr(self):
        return "%d, heads=%d, key_heads=%d, dk=%d, dv=%d" % (self.dim, self.heads, self.key_heads, self.dk, self.dv)
