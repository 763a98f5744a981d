"""Measured cases of the operators that a delta-rule mixer has beside linear
attention: the gated delta rule (prompt, backward, single token) and the norm
of queries and keys for each head with the position rotation in the same pass
(forward, backward).

`own` selects the framework's kernels; otherwise `run` computes the same
results from elementary torch operations in 32 bits, rounded once at the end.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
CHUNK = 64  # positions a chunk of the plain delta rule


def listed():
    return [
        # a short prompt of one user: latency
        {"name": "delta_prompt_short", "op": "delta_forward", "dtype": "bf16", "B": 1, "L": 64, "H": 16, "Hk": 16,
         "dk": 64, "dv": 64, "state": False},
        # a training batch's forward pass
        {"name": "delta_train_fwd", "op": "delta_forward", "dtype": "bf16", "B": 8, "L": 2048, "H": 16, "Hk": 16,
         "dk": 128, "dv": 128, "state": False},
        # one long document continued from a state: few rows, a long axis, an odd length
        {"name": "delta_document", "op": "delta_forward", "dtype": "f32", "B": 1, "L": 32771, "H": 8, "Hk": 8,
         "dk": 64, "dv": 128, "state": True},
        # the training batch's backward pass
        {"name": "delta_train_bwd", "op": "delta_backward", "dtype": "bf16", "B": 8, "L": 2048, "H": 16, "Hk": 16,
         "dk": 128, "dv": 128, "state": False},
        # fp32 training (this framework's own type): ragged length, odd head sizes, two heads sharing a key, a state
        {"name": "delta_bwd_ragged", "op": "delta_backward", "dtype": "f32", "B": 3, "L": 1000, "H": 10, "Hk": 5,
         "dk": 48, "dv": 80, "state": True},
        # single-token decoding of one user: latency
        {"name": "delta_step_one", "op": "delta_step", "dtype": "bf16", "B": 1, "H": 16, "Hk": 16, "dk": 128,
         "dv": 128},
        # single-token decoding of a full serving batch
        {"name": "delta_step_batch", "op": "delta_step", "dtype": "bf16", "B": 128, "H": 16, "Hk": 16, "dk": 128,
         "dv": 128},
        # the training batch's queries and keys, weighted norm and full rotation
        {"name": "headnorm_fwd_train", "op": "headnorm_forward", "dtype": "bf16", "B": 8, "L": 2048, "Hq": 16,
         "Hk": 16, "d": 128, "R": 128, "kind": "rms", "weight": True, "interleaved": False},
        # one token of one user, half of each head rotated: latency
        {"name": "headnorm_fwd_token", "op": "headnorm_forward", "dtype": "bf16", "B": 1, "L": 1, "Hq": 16, "Hk": 16,
         "d": 128, "R": 64, "kind": "rms", "weight": True, "interleaved": False},
        # the training batch's backward pass
        {"name": "headnorm_bwd_train", "op": "headnorm_backward", "dtype": "bf16", "B": 8, "L": 2048, "Hq": 16,
         "Hk": 16, "d": 128, "R": 128, "kind": "rms", "weight": True, "interleaved": False},
        # fp32 training of the delta rule: unit lengths, no rotation, fewer key heads, odd sizes
        {"name": "headnorm_bwd_ragged", "op": "headnorm_backward", "dtype": "f32", "B": 3, "L": 1000, "Hq": 10,
         "Hk": 5, "d": 48, "R": 0, "kind": "l2", "weight": False, "interleaved": False},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["delta_forward", "delta_forward", "delta_backward", "delta_backward", "delta_step",
                     "headnorm_forward", "headnorm_backward"])
    c = {"op": op, "dtype": rng.choice(["f32", "bf16"])}
    if op.startswith("delta"):
        c["dk"] = rng.choice([16, 32, 48, 64, 64, 80, 96, 128, 128, rng.randint(8, 128)])
        c["dv"] = rng.choice([16, 32, 48, 64, 64, 80, 96, 128, 128, rng.randint(8, 128)])
        group = rng.choice([1, 1, 1, 2, 4])
        c["Hk"] = rng.randint(1, 32 // group)
        if op == "delta_step":
            c["B"] = _log_int(rng, 1, 128)
            while c["B"] * c["Hk"] * group > 2048:
                c["B"] = max(1, c["B"] // 2)
        else:
            c["L"] = _log_int(rng, 1, 32768)
            c["B"] = _log_int(rng, 1, 16)
            c["state"] = rng.random() < 0.5
            most = 8 * 2048 * 16 // (1 if c["dtype"] == "bf16" else 2)
            while c["B"] * c["L"] * c["Hk"] * group > most:
                if c["B"] > 1:
                    c["B"] //= 2
                elif c["Hk"] * group > 8:
                    c["Hk"] = (c["Hk"] + 1) // 2
                else:
                    c["L"] //= 2
        c["H"] = c["Hk"] * group
        return c
    c["B"], c["L"] = _log_int(rng, 1, 16), _log_int(rng, 1, 32768)
    c["Hk"] = rng.randint(1, 16)
    c["Hq"] = c["Hk"] * rng.choice([1, 1, 2, 4])
    c["d"] = 2 * rng.choice([16, 32, 40, 64, 64, rng.randint(4, 64)])
    c["R"] = rng.choice([0, c["d"], c["d"], 2 * rng.randint(1, c["d"] // 2)])
    c["kind"] = rng.choice(["rms", "rms", "l2"])
    c["weight"] = rng.random() < 0.7
    c["interleaved"] = rng.random() < 0.3
    most = 8 * 2048 * 32 * 128 // (1 if c["dtype"] == "bf16" else 2)
    while c["B"] * c["L"] * (c["Hq"] + c["Hk"]) * c["d"] > most:
        if c["B"] > 1:
            c["B"] //= 2
        else:
            c["L"] //= 2
    return c


# ---------------------------------------------------------------- inputs
EPS = 1e-6


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    T = TYPES[case["dtype"]]

    def normal(*shape, dtype=T, std=1.0):
        return (torch.randn(*shape, generator=gen, device=DEV) * std).to(dtype)

    def unit(*shape):
        x = torch.randn(*shape, generator=gen, device=DEV)
        return (x * torch.rsqrt((x * x).sum(-1, keepdim=True) + EPS)).to(T)

    op, B = case["op"], case["B"]
    s = {"case": case}
    if op.startswith("delta"):
        H, Hk, dk, dv = (case[k] for k in ("H", "Hk", "dk", "dv"))
        seq = () if op == "delta_step" else (case["L"],)
        s["q"], s["k"], s["v"] = unit(B, *seq, Hk, dk), unit(B, *seq, Hk, dk), normal(B, *seq, H, dv)
        # memories from a few positions to some thousands, spread over the heads, and varying from token to token
        rate = torch.exp2(-11.0 * (torch.arange(H, device=DEV) + torch.rand(H, generator=gen, device=DEV)) / H)
        s["log_decay"] = -rate * torch.nn.functional.softplus(normal(B, *seq, H, dtype=torch.float32))
        s["beta"] = torch.sigmoid(normal(B, *seq, H, dtype=torch.float32))
        s["state"] = None
        if op == "delta_step" or case["state"]:
            s["state"] = normal(B, H, dk, dv, dtype=torch.float32)
        if op == "delta_step":
            s["next"] = torch.empty_like(s["state"])  # where the next token's call finds its state
        if op == "delta_backward":
            s["grad_o"] = normal(B, *seq, H, dv)
            s["grad_state"] = normal(B, H, dk, dv, dtype=torch.float32) if case["state"] else None
        return s
    L, Hq, Hk, d, R = (case[k] for k in ("L", "Hq", "Hk", "d", "R"))
    s["q"], s["k"] = normal(B, L, Hq, d), normal(B, L, Hk, d, std=2.0)
    s["wq"] = s["wk"] = s["table"] = s["positions"] = None
    if case["weight"]:
        s["wq"], s["wk"] = (1.0 + normal(d, dtype=torch.float32, std=0.1) for _ in range(2))
    if R:
        # cosines and sines of a context's positions; each row of the batch stands somewhere in it
        n = L + 4096
        angle = torch.arange(n, device=DEV, dtype=torch.float64)[:, None] * 10000.0 ** (
            -torch.arange(0, R, 2, device=DEV, dtype=torch.float64) / R)
        s["table"] = torch.cat([angle.cos(), angle.sin()], 1).float()
        start = torch.randint(0, 4096, (B, 1), generator=gen, device=DEV)
        s["positions"] = start + torch.arange(L, device=DEV)
    if op == "headnorm_backward":
        s["gq"], s["gk"] = normal(B, L, Hq, d), normal(B, L, Hk, d)
        for n in "qk":
            x = s[n].float()
            m = (x * x).sum(-1) if case["kind"] == "l2" else (x * x).mean(-1)
            s["r" + n] = torch.rsqrt(m + EPS)
    return s


# ---------------------------------------------------------------- plain delta rule
def _chunks(x, nc):
    """[B, L, H, d] as fp32 chunks [nc, B, H, CHUNK, d], zeros past the end."""
    B, L, H, d = x.shape
    x = torch.nn.functional.pad(x.float(), (0, 0, 0, 0, 0, nc * CHUNK - L))
    return x.view(B, nc, CHUNK, H, d).permute(1, 0, 3, 2, 4).contiguous()


def _tokens(x, L):
    """The inverse of _chunks."""
    nc, B, H, _, d = x.shape
    return x.permute(1, 0, 3, 2, 4).reshape(B, nc * CHUNK, H, d)[:, :L]


def _t(x):
    return x.transpose(-1, -2).contiguous()


def _shared(x, H):
    """Heads of queries or keys, repeated for the heads of values that share them."""
    return x.repeat_interleave(H // x.shape[-2], -2)


def _parts(s):
    """The chunks' operands: q, k, v, decays from position to position E, from the chunk's start f and to its end r,
    beta, the inverse T of I + A, and the whole chunk's decay."""
    H, L = s["case"]["H"], s["case"]["L"]
    nc = -(-L // CHUNK)
    q, k, v = _chunks(_shared(s["q"], H), nc), _chunks(_shared(s["k"], H), nc), _chunks(s["v"], nc)
    beta = _chunks(s["beta"][..., None], nc)
    G = _chunks(s["log_decay"][..., None], nc)[..., 0].double().cumsum(-1)   # differences of long sums
    lower = torch.ones(CHUNK, CHUNK, device=DEV).tril()
    E = torch.exp((G[..., :, None] - G[..., None, :]).clamp(max=0.0)).float() * lower
    f, r = torch.exp(G).float()[..., None], torch.exp(G[..., -1:] - G).float()[..., None]
    eye = torch.eye(CHUNK, device=DEV)
    a = (k @ _t(k)) * (E - eye)
    # (I + A)^-1 = (I - A)(I + A^2)(I + A^4) ...: A is strictly lower triangular
    A = beta * a
    T, power = eye - A, A @ A
    for _ in range(5):
        T, power = T + T @ power, power @ power
    return q, k, v, beta, E, f, r, f[..., -1:, :], a, T


def _initial(s):
    c = s["case"]
    return torch.zeros(c["B"], c["H"], c["dk"], c["dv"], device=DEV) if s["state"] is None else s["state"]


def _plain_delta(s):
    q, k, v, beta, E, f, r, whole, _, T = _parts(s)
    S, o = _initial(s), torch.empty_like(v)
    P = (q @ _t(k)) * E
    kr, kf, qf, Tb = _t(k * r), k * f, q * f, T * _t(beta)
    for c in range(q.shape[0]):
        u = Tb[c] @ (v[c] - kf[c] @ S)
        o[c] = qf[c] @ S + P[c] @ u
        S = whole[c] * S + kr[c] @ u
    o = _tokens(o, s["case"]["L"]) * s["case"]["dk"] ** -0.5
    return o.to(s["q"].dtype).contiguous(), S


def _plain_delta_backward(s):
    q, k, v, beta, E, f, r, whole, a, T = _parts(s)
    c = s["case"]
    nc = q.shape[0]
    do = _chunks(s["grad_o"], nc) * c["dk"] ** -0.5
    P = (q @ _t(k)) * E
    kr, kf, qf, Tb, Pt, Tt = k * r, k * f, q * f, T * _t(beta), _t(P), _t(T)
    krt, kft, qft = _t(kr), _t(kf), _t(qf)
    S = _initial(s)
    before, after, w, u, dR = [], [None] * nc, torch.empty_like(v), torch.empty_like(v), torch.empty_like(v)
    for i in range(nc):
        before.append(S)
        w[i] = v[i] - kf[i] @ S
        u[i] = Tb[i] @ w[i]
        S = whole[i] * S + krt[i] @ u[i]
    D = torch.zeros_like(S) if s["grad_state"] is None else s["grad_state"]
    for i in reversed(range(nc)):
        after[i] = D
        dR[i] = Tt[i] @ (Pt[i] @ do[i] + kr[i] @ D)
        D = whole[i] * D + qft[i] @ do[i] - kft[i] @ (beta[i] * dR[i])
    S0, D1 = torch.stack(before), torch.stack(after)
    dr = beta * dR
    dP, dA = do @ _t(u) * E, -(dr @ _t(u)) * (E - torch.eye(CHUNK, device=DEV))
    toS, fromS, fromD = f * (do @ _t(S0)), f * (dr @ _t(S0)), r * (u @ _t(D1))
    dq = toS + dP @ k
    dk = fromD - fromS + _t(dP) @ q + (dA + _t(dA)) @ k
    dbeta = (dR * w).sum(-1) - ((dR @ _t(u)) * a).sum(-1)
    # a gate stands between every earlier and every later position of its chunk
    y, x = (q * toS).sum(-1) - (k * fromS).sum(-1), (k * fromD).sum(-1)
    pairs = dP * (q @ _t(k)) * (1 - torch.eye(CHUNK, device=DEV)) + dA * (k @ _t(k))
    # (all pairs that end at or after it, less those that also begin there)
    y = (y + pairs.sum(-1) - pairs.sum(-2)).double()
    total = whole[..., 0] * (D1 * S0).sum((-1, -2))[..., None]
    dg = (total + y.flip(-1).cumsum(-1).flip(-1) + x.double().cumsum(-1) - x).float()
    L, Hk, H = c["L"], c["Hk"], c["H"]
    dq, dk = (_tokens(t, L).unflatten(2, (Hk, H // Hk)).sum(3) for t in (dq, dk))
    T_ = s["q"].dtype
    out = [dq.to(T_).contiguous(), dk.to(T_).contiguous(), _tokens(dr, L).to(T_).contiguous(),
           _tokens(dg[..., None], L)[..., 0].contiguous(), _tokens(dbeta[..., None], L)[..., 0].contiguous()]
    return out + ([D] if s["state"] is not None else [])


def _plain_delta_step(s):
    H = s["case"]["H"]
    q, k = (_shared(s[n], H).float() for n in "qk")
    S = torch.exp(s["log_decay"])[..., None, None] * s["state"]
    u = s["beta"][..., None] * (s["v"].float() - (k[..., :, None] * S).sum(-2))
    new = S + k[..., :, None] * u[..., None, :]
    o = (q[..., :, None] * new).sum(-2) * q.shape[-1] ** -0.5
    return o.to(s["q"].dtype), new


# ---------------------------------------------------------------- plain norm and rotation
def _halves(x, interleaved):
    """The two numbers of each rotated pair."""
    return (x[..., 0::2], x[..., 1::2]) if interleaved else x.chunk(2, -1)


def _whole(a, b, interleaved):
    return torch.stack([a, b], -1).flatten(-2) if interleaved else torch.cat([a, b], -1)


def _rotate(x, s, sign):
    R = s["case"]["R"]
    if R == 0:
        return x
    rows = s["table"].to(x.dtype)[s["positions"]][:, :, None]
    cos, sin = rows[..., :R // 2], sign * rows[..., R // 2:]
    a, b = _halves(x[..., :R], s["case"]["interleaved"])
    return torch.cat([_whole(a * cos - b * sin, b * cos + a * sin, s["case"]["interleaved"]), x[..., R:]], -1)


def _mean(x, case):
    return x.sum(-1, keepdim=True) if case["kind"] == "l2" else x.mean(-1, keepdim=True)


def _plain_headnorm(s):
    out = []
    for x, w in ((s["q"], s["wq"]), (s["k"], s["wk"])):
        f = x.float()
        r = torch.rsqrt(_mean(f * f, s["case"]) + EPS)
        y = f * r if w is None else f * r * w
        out += [_rotate(y, s, 1.0).to(x.dtype), r[..., 0]]
    return out[0], out[2], out[1], out[3]


def _plain_headnorm_backward(s):
    out, weights = [], []
    for x, r, g, w in ((s["q"], s["rq"], s["gq"], s["wq"]), (s["k"], s["rk"], s["gk"], s["wk"])):
        r = r[..., None]
        xh = x.float() * r
        dy = _rotate(g.float(), s, -1.0)
        weights += [] if w is None else [(dy * xh).double().sum((0, 1, 2)).float()]
        dy = dy if w is None else dy * w
        out.append((r * (dy - xh * _mean(dy * xh, s["case"]))).to(x.dtype))
    return out + weights


PLAIN = {"delta_forward": _plain_delta, "delta_backward": _plain_delta_backward, "delta_step": _plain_delta_step,
         "headnorm_forward": _plain_headnorm, "headnorm_backward": _plain_headnorm_backward}


# ---------------------------------------------------------------- the framework's calls
def _own(s):
    from nonlinear_rnn_solve_pararnn_amd import api
    op = s["case"]["op"]
    if op == "delta_forward":
        return api.delta_forward(s["q"], s["k"], s["v"], s["log_decay"], s["beta"], s["state"])
    if op == "delta_backward":
        out = api.delta_backward(s["q"], s["k"], s["v"], s["log_decay"], s["beta"], s["grad_o"], s["state"],
                                 s["grad_state"])
        return list(out if s["state"] is not None else out[:5])
    if op == "delta_step":
        return api.delta_step(s["q"], s["k"], s["v"], s["log_decay"], s["beta"], s["state"], out_state=s["next"])
    kw = {"kind": s["case"]["kind"], "interleaved": s["case"]["interleaved"]}
    if op == "headnorm_forward":
        return api.headnorm_forward(s["q"], s["k"], s["wq"], s["wk"], s["table"], s["positions"], eps=EPS, **kw)
    out = api.headnorm_backward(s["q"], s["k"], s["rq"], s["rk"], s["gq"], s["gk"], s["wq"], s["wk"], s["table"],
                                s["positions"], **kw)
    return list(out if s["wq"] is not None else out[:2])


def run(state):
    if own:
        return _own(state)
    return PLAIN[state["case"]["op"]](state)


def work(case):
    op, e = case["op"], 2 if case["dtype"] == "bf16" else 4
    if op.startswith("delta"):
        B, H, Hk, dk, dv = (case[k] for k in ("B", "H", "Hk", "dk", "dv"))
        state = 4 * B * H * dk * dv
        if op == "delta_step":
            return {"bytes": 2 * state + B * (2 * Hk * dk + 2 * H * dv) * e + 8 * B * H, "flops": 7 * B * H * dk * dv}
        n = B * case["L"]
        # the state's product with the key, its update and its product with the query, 2 dk dv each, a token
        if op == "delta_forward":
            return {"bytes": n * ((2 * Hk * dk + 2 * H * dv) * e + 8 * H) + state * (2 if case["state"] else 1),
                    "flops": 6 * n * H * dk * dv}
        return {"bytes": n * ((4 * Hk * dk + 3 * H * dv) * e + 16 * H) + (3 * state if case["state"] else 0),
                "flops": 18 * n * H * dk * dv}
    rows = case["B"] * case["L"]
    n = rows * (case["Hq"] + case["Hk"])
    turn = min(rows, case["L"] + 4096) * case["R"] * 4 + (8 * rows if case["R"] else 0)
    weights = 8 * case["d"] if case["weight"] else 0
    if op == "headnorm_forward":
        return {"bytes": 2 * n * case["d"] * e + 4 * n + turn + weights, "flops": 8 * n * case["d"]}
    return {"bytes": 3 * n * case["d"] * e + 4 * n + turn + 2 * weights, "flops": 14 * n * case["d"]}


# ---------------------------------------------------------------- 64 bits
def _states(f, start, first, count, keep):
    """The recurrence itself from `start`, position by position: states, errors w and outputs of positions
    first .. first + count - 1 (the states only if they are to be kept)."""
    S, states, ws, outs = start, [], [], []
    for t in range(first, first + count):
        if keep:
            states.append(S)
        S = f["decay"][:, t] * S
        w = f["v"][:, t] - (f["k"][:, t, :, :, None] * S).sum(-2)
        S = S + f["k"][:, t, :, :, None] * (f["beta"][:, t] * w)[:, :, None]
        ws.append(w)
        if not keep:
            outs.append((f["q"][:, t, :, :, None] * S).sum(-2))
    return S, states, ws, outs


def _exact_delta(s, case):
    back, H, L = case["op"] == "delta_backward", case["H"], 1 if case["op"] == "delta_step" else case["L"]
    f = {n: _shared(s[n], H) if n in "qk" else s[n] for n in ("q", "k", "v", "log_decay", "beta")}
    if case["op"] == "delta_step":
        f = {n: t[:, None] for n, t in f.items()}
    f = {n: t.double() for n, t in f.items()}
    f["decay"] = torch.exp(f["log_decay"])[..., None, None]
    f["beta"] = f["beta"][..., None]
    S = _initial(s).double()
    scale = case["dk"] ** -0.5
    if not back:
        S, _, _, outs = _states(f, S, 0, L, False)
        o = torch.stack(outs, 1) * scale
        return (o[:, 0] if case["op"] == "delta_step" else o), S
    # states at the segments' starts, then each segment again with all of its states
    seg = max(1, math.isqrt(L))
    starts = []
    for t in range(0, L, seg):
        starts.append(S)
        S = _states(f, S, t, min(seg, L - t), False)[0]
    D = torch.zeros_like(S) if s["grad_state"] is None else s["grad_state"].double()
    do = s["grad_o"].double() * scale
    out = {n: [None] * L for n in ("q", "k", "v", "g", "b")}
    for n, t0 in reversed(list(enumerate(range(0, L, seg)))):
        _, states, ws, _ = _states(f, starts[n], t0, min(seg, L - t0), True)
        for t in reversed(range(t0, t0 + len(ws))):
            k, q, b, w = f["k"][:, t], f["q"][:, t], f["beta"][:, t], ws[t - t0]
            S0 = f["decay"][:, t] * states[t - t0]
            u = b * w
            D = D + q[..., :, None] * do[:, t, :, None]
            out["q"][t] = ((S0 + k[..., :, None] * u[:, :, None]) * do[:, t, :, None]).sum(-1)
            du = (k[..., :, None] * D).sum(-2)
            dw = b * du
            out["v"][t], out["b"][t] = dw, (du * w).sum(-1)
            out["k"][t] = (D * u[:, :, None]).sum(-1) - (S0 * dw[:, :, None]).sum(-1)
            D = D - k[..., :, None] * dw[:, :, None]
            out["g"][t] = (D * S0).sum((-1, -2))
            D = f["decay"][:, t] * D
    out = {n: torch.stack(t, 1) for n, t in out.items()}
    for n in "qk":
        out[n] = out[n].unflatten(2, (case["Hk"], H // case["Hk"])).sum(3)
    return [out[n] for n in ("q", "k", "v", "g", "b")] + ([D] if s["state"] is not None else [])


def _exact_turn(x, s, case, back):
    """x's pairs as complex numbers, turned by their positions' angles (or back)."""
    R = case["R"]
    if R == 0:
        return x
    row = s["table"][s["positions"].long()].double()[:, :, None]
    turn = torch.complex(row[..., :R // 2], -row[..., R // 2:] if back else row[..., R // 2:])
    first, second = (torch.arange(R // 2, device=DEV) * 2, torch.arange(R // 2, device=DEV) * 2 + 1) \
        if case["interleaved"] else (torch.arange(R // 2, device=DEV), torch.arange(R // 2, device=DEV) + R // 2)
    z = torch.complex(x[..., first], x[..., second]) * turn
    y = x.clone()
    y[..., first], y[..., second] = z.real, z.imag
    return y


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"].startswith("delta"):
        return _exact_delta(s, case)
    first, second = [], []
    for n in "qk":
        x, w = s[n].double(), 1.0 if s["w" + n] is None else s["w" + n].double()
        count = 1 if case["kind"] == "l2" else case["d"]
        if case["op"] == "headnorm_forward":
            r = 1.0 / torch.sqrt(x.square().sum(-1) / count + EPS)
            first.append(_exact_turn(x * r[..., None] * w, s, case, False))
            second.append(r)
        else:
            r = s["r" + n].double()[..., None]
            g = _exact_turn(s["g" + n].double(), s, case, True)
            gx = g * w * r
            first.append(gx - x * r * r * (gx * x).sum(-1, keepdim=True) / count)
            if case["weight"]:
                second.append((g * x * r).sum((0, 1, 2)))
    return first + second
