"""Plain fp64 references of the operators around the recurrences, written from
their formulas on CPU tensors: the recurrence position by position, row
statistics, and a loop over tokens."""
import torch


def f64(*ts):
    return [None if t is None else t.detach().cpu().double() for t in ts]


def linattn(q, k, v, g, state=None, scale=None):
    """(o, final state); q, k [B, L, H, dk], v [B, L, H, dv], g [H]."""
    B, L, H, dk = q.shape
    scale = dk ** -0.5 if scale is None else scale
    lam = torch.exp(g).view(1, H, 1, 1)
    S = torch.zeros(B, H, dk, v.shape[-1], dtype=q.dtype) if state is None else state
    o = []
    for t in range(L):
        S = lam * S + k[:, t, :, :, None] * v[:, t, :, None, :]
        o.append(scale * (q[:, t, :, :, None] * S).sum(-2))
    return torch.stack(o, 1), S


def linattn_grads(q, k, v, g, do, state=None, grad_state=None, scale=None):
    """(dq, dk, dv, dstate) by the adjoint recurrence."""
    B, L, H, dk = q.shape
    scale = dk ** -0.5 if scale is None else scale
    lam = torch.exp(g).view(1, H, 1, 1)
    S = torch.zeros(B, H, dk, v.shape[-1], dtype=q.dtype) if state is None else state
    dq, gk, gv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    for t in range(L):
        S = lam * S + k[:, t, :, :, None] * v[:, t, :, None, :]
        dq[:, t] = scale * (S * do[:, t, :, None, :]).sum(-1)
    D = torch.zeros_like(S) if grad_state is None else grad_state
    for t in range(L - 1, -1, -1):
        D = D + scale * q[:, t, :, :, None] * do[:, t, :, None, :]
        gk[:, t] = (D * v[:, t, :, None, :]).sum(-1)
        gv[:, t] = (D * k[:, t, :, :, None]).sum(-2)
        D = lam * D
    return dq, gk, gv, D


def layernorm(s, w=None, b=None, eps=1e-5):
    """(y, mean, rstd)."""
    mean = s.sum(-1, keepdim=True) / s.shape[-1]
    var = ((s - mean) ** 2).sum(-1, keepdim=True) / s.shape[-1]
    rstd = 1.0 / torch.sqrt(var + eps)
    y = (s - mean) * rstd
    if w is not None:
        y = y * w
    if b is not None:
        y = y + b
    return y, mean[..., 0], rstd[..., 0]


def layernorm_grads(s, w, mean, rstd, dy, ds=None):
    """(dx, dw, db)."""
    xh = (s - mean[..., None]) * rstd[..., None]
    g = dy if w is None else dy * w
    D = s.shape[-1]
    dx = rstd[..., None] * (g - g.sum(-1, keepdim=True) / D - xh * (g * xh).sum(-1, keepdim=True) / D)
    if ds is not None:
        dx = dx + ds
    return dx, (dy * xh).reshape(-1, D).sum(0), dy.reshape(-1, D).sum(0)


def embedding_grad(ids, grad, V, scale=1.0, padding_idx=None):
    out = torch.zeros(V, grad.shape[-1], dtype=grad.dtype)
    for i, r in zip(ids.reshape(-1).tolist(), grad.reshape(-1, grad.shape[-1])):
        if 0 <= i < V and i != padding_idx:
            out[i] += r
    return out * scale


def rel(got, ref):
    """2-norm of the difference over the 2-norm of the reference."""
    got, ref = got.detach().cpu().double(), ref.double()
    assert got.shape == ref.shape, (got.shape, ref.shape)
    d = float((got - ref).norm())
    n = float(ref.norm())
    return d / n if n > 0 else d
