"""Plain fp64 references of the delta-rule mixer's operators, written from
their formulas on CPU tensors: the recurrence position by position with its
adjoint, and row norms with the rotation."""
import torch


def heads(x, H):
    """Heads of queries or keys, repeated for the heads of values that share them."""
    return x.repeat_interleave(H // x.shape[-2], -2)


def delta(q, k, v, g, b, state=None, scale=None):
    """(o, final state); q, k [B, L, Hk, dk], v [B, L, H, dv], g, b [B, L, H]."""
    (B, L, H, dv), dk = v.shape, q.shape[-1]
    scale = dk ** -0.5 if scale is None else scale
    q, k = heads(q, H), heads(k, H)
    S = torch.zeros(B, H, dk, dv, dtype=q.dtype) if state is None else state
    o = []
    for t in range(L):
        S = torch.exp(g[:, t])[..., None, None] * S
        kt = k[:, t, :, :, None]
        u = b[:, t, :, None] * (v[:, t] - (kt * S).sum(-2))
        S = S + kt * u[:, :, None]
        o.append(scale * (q[:, t, :, :, None] * S).sum(-2))
    return torch.stack(o, 1), S


def delta_grads(q, k, v, g, b, do, state=None, grad_state=None, scale=None):
    """(dq, dk, dv, dg, db, dstate) by the adjoint recurrence."""
    (B, L, H, dv), dk, Hk = v.shape, q.shape[-1], q.shape[-2]
    scale = dk ** -0.5 if scale is None else scale
    q, k = heads(q, H), heads(k, H)
    S = torch.zeros(B, H, dk, dv, dtype=q.dtype) if state is None else state
    decayed, errors = [], []
    for t in range(L):
        S = torch.exp(g[:, t])[..., None, None] * S
        decayed.append(S)
        kt = k[:, t, :, :, None]
        errors.append(v[:, t] - (kt * S).sum(-2))
        S = S + kt * (b[:, t, :, None] * errors[-1])[:, :, None]
    D = torch.zeros_like(S) if grad_state is None else grad_state
    gq, gk, gv, gg, gb = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v), torch.empty_like(g), torch.empty_like(b)
    for t in range(L - 1, -1, -1):
        kt, dot, S0, w = k[:, t, :, :, None], scale * do[:, t, :, None, :], decayed[t], errors[t]
        u = b[:, t, :, None] * w
        S1 = S0 + kt * u[:, :, None]
        gq[:, t] = (S1 * dot).sum(-1)
        D = D + q[:, t, :, :, None] * dot
        du = (kt * D).sum(-2)
        gb[:, t] = (du * w).sum(-1)
        gv[:, t] = b[:, t, :, None] * du
        gk[:, t] = (D * u[:, :, None]).sum(-1) - (S0 * gv[:, t, :, None, :]).sum(-1)
        D = D - kt * gv[:, t, :, None, :]
        gg[:, t] = (D * S0).sum((-1, -2))
        D = torch.exp(g[:, t])[..., None, None] * D
    gq, gk = (x.unflatten(2, (Hk, H // Hk)).sum(3) for x in (gq, gk))
    return gq, gk, gv, gg, gb, D


def table(P, R, base=10000.0):
    """[P, R]: cosines, then sines of P positions."""
    angle = torch.arange(P, dtype=torch.float64)[:, None] * base ** (-torch.arange(0, R, 2, dtype=torch.float64) / R)
    return torch.cat([angle.cos(), angle.sin()], 1)


def turn(x, tab, positions, interleaved, back=False):
    """The first R elements of x [B, L, H, d] as complex numbers, turned by their position's angles (or back)."""
    if tab is None:
        return x
    R = tab.shape[1]
    row = tab[positions][:, :, None]
    e = torch.complex(row[..., :R // 2], -row[..., R // 2:] if back else row[..., R // 2:])
    i = torch.arange(R // 2)
    first, second = (2 * i, 2 * i + 1) if interleaved else (i, i + R // 2)
    z = torch.complex(x[..., first], x[..., second]) * e
    y = x.clone()
    y[..., first], y[..., second] = z.real, z.imag
    return y


def headnorm(x, w, tab, positions, kind="rms", eps=1e-6, interleaved=False):
    """(y, r) of x [B, L, H, d]."""
    m = (x * x).sum(-1) / (x.shape[-1] if kind == "rms" else 1)
    r = 1.0 / torch.sqrt(m + eps)
    n = x * r[..., None]
    if w is not None:
        n = n * w
    return turn(n, tab, positions, interleaved), r


def headnorm_grads(x, r, dy, w, tab, positions, kind="rms", interleaved=False):
    """(dx, dw)."""
    xh = x * r[..., None]
    g = turn(dy, tab, positions, interleaved, back=True)
    dw = (g * xh).reshape(-1, x.shape[-1]).sum(0)
    if w is not None:
        g = g * w
    m = (g * xh).sum(-1, keepdim=True) / (x.shape[-1] if kind == "rms" else 1)
    return r[..., None] * (g - xh * m), dw
