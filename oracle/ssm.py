"""fp64 oracle of the short causal convolution and of the selective scan -- TEST
INFRASTRUCTURE.

numpy, token by token in the order of the definitions, sharing no code with the
library; gradients are the reverse of these lines.

    u_t = bias + sum_j w[c,j] x_{t-W+1+j},           y_t = act(u_t)
    S_t = exp(dt_t A) S_{t-1} + dt_t x_t B_t,        dt_t = softplus(delta_t + bias)
    out_t = (sum_s C_t S_t + D x_t) z_t sigmoid(z_t)

``plant`` names one deliberate mistake, for the tests that prove the pins catch it.
"""
from __future__ import annotations

import numpy as np


def _f(x):
    return None if x is None else np.asarray(x, np.float64)


def _sigmoid(u):
    e = np.exp(-np.abs(u))
    return np.where(u >= 0, 1.0, e) / (1.0 + e)


def act(u, activation):
    """Value and slope."""
    if activation == "none":
        return u, np.ones_like(u)
    s = _sigmoid(u)
    slope = s * _sigmoid(-u)
    return (s, slope) if activation == "sigmoid" else (u * s, s + u * slope)


def softplus(u):
    """Value and slope."""
    return np.maximum(u, 0.0) + np.log1p(np.exp(-np.abs(u))), _sigmoid(u)


def _ends(lengths, B, N):
    return np.full(B, N) if lengths is None else np.clip(np.asarray(lengths).astype(int), 0, N)


def conv(x, weight, bias=None, *, activation="silu", S0=None, lengths=None, dy=None, dS_out=None, plant=None):
    """(y [B,N,C], window), or for dy (y, window, dx, dweight, dbias, dS0)."""
    x, w = _f(x), _f(weight)
    B, N, C = x.shape
    W = w.shape[1]
    b = np.zeros(C) if bias is None else _f(bias)
    seen = np.zeros((B, W - 1 + N, C))
    if S0 is not None:
        seen[:, :W - 1] = _f(S0)
    seen[:, W - 1:] = x
    if plant == "taps_reversed":
        w = w[:, ::-1]
    y, window = np.zeros((B, N, C)), np.zeros((B, W - 1, C))
    dseen, dw, db = np.zeros_like(seen), np.zeros((C, W)), np.zeros(C)
    for r, end in enumerate(_ends(lengths, B, N)):
        window[r] = seen[r, N:] if plant == "window_ignores_length" else seen[r, end:end + W - 1]
        if dS_out is not None:
            dseen[r, end:end + W - 1] += _f(dS_out)[r]
        for t in range(end):
            u = b + (w.T * seen[r, t:t + W]).sum(0)
            y[r, t], slope = act(u, activation)
            if dy is not None:
                du = _f(dy)[r, t] * (1.0 if plant == "no_slope" else slope)
                db += du
                dw += (du * seen[r, t:t + W]).T
                dseen[r, t:t + W] += w.T * du
    if dy is None:
        return y, window
    return y, window, dseen[:, W - 1:], dw, db, dseen[:, :W - 1]


def scan(x, delta, A, Bm, Cm, *, D=None, z=None, delta_bias=None, softplus_on=True, S0=None, lengths=None,
         dout=None, dS_out=None, plant=None):
    """(out, S), or for dout a dict of out, S and the gradients under the names of the inputs."""
    x, delta, A, Bm, Cm = _f(x), _f(delta), _f(A), _f(Bm), _f(Cm)
    B, N, C = x.shape
    G, n = Bm.shape[2:]
    d_skip = np.zeros(C) if D is None else _f(D)
    pre = delta + (0.0 if delta_bias is None else _f(delta_bias))
    dt, slope = softplus(pre) if softplus_on else (pre, np.ones_like(pre))
    gate, gate_slope = act(_f(z), "silu") if z is not None else (np.ones_like(x), np.zeros_like(x))
    wide = lambda r: np.repeat(r, C // G, axis=1)  # noqa: E731  [B,G,n] -> [B,C,n]
    ends = _ends(lengths, B, N)
    S = np.zeros((B, C, n)) if S0 is None else _f(S0).copy()
    out, kept = np.zeros((B, N, C)), []
    for t in range(N):
        on = (t < ends)[:, None]
        held = np.exp(dt[:, t, :, None] * A) * S
        if plant == "undecayed":
            held = S
        new = held + (dt[:, t] * x[:, t])[..., None] * wide(Bm[:, t])
        if plant == "input_not_stepped":
            new = held + x[:, t, :, None] * wide(Bm[:, t])
        read = S if plant == "read_before_write" else new
        kept.append((held, new))
        S = np.where(on[..., None], new, S)
        y = (read * wide(Cm[:, t])).sum(-1) + d_skip * x[:, t]
        out[:, t] = np.where(on, y * gate[:, t], 0.0)
    if dout is None:
        return out, S
    g = {k: np.zeros_like(v) for k, v in dict(x=x, delta=x, A=A, Bm=Bm, Cm=Cm, D=d_skip, z=x).items()}
    g["delta_bias"] = np.zeros(C)
    dS = np.zeros_like(S) if dS_out is None else _f(dS_out).copy()
    group = lambda r: r.reshape(B, G, C // G, n).sum(2)  # noqa: E731
    for t in reversed(range(N)):
        on = (t < ends)[:, None]
        held, new = kept[t]
        # behind a row's end every input is zero, and the states of its last token are not read
        live = lambda v: np.where(on if v.ndim == 2 else on[..., None], v, 0.0)  # noqa: E731
        held, new, do, xt, dtt = map(live, (held, new, _f(dout)[:, t], x[:, t], dt[:, t]))
        Bt, Ct = live(wide(Bm[:, t])), live(wide(Cm[:, t]))
        y = (new * Ct).sum(-1) + d_skip * xt
        g["z"][:, t] = do * y * live(gate_slope[:, t])
        dy = do * live(gate[:, t])
        g["Cm"][:, t] = group(dy[..., None] * new)
        dS = dS + dy[..., None] * Ct
        here = live(dS)
        q = here * (new if plant == "decay_of_the_new_state" else held)
        w = (here * Bt).sum(-1)
        g["Bm"][:, t] = group(here * (dtt * xt)[..., None])
        g["A"] += (q * dtt[..., None]).sum(0)
        g["x"][:, t] = w * dtt + d_skip * dy
        g["D"] += (dy * xt).sum(0)
        g["delta"][:, t] = (q * A).sum(-1) + w * xt
        if plant != "softplus_not_differentiated":
            g["delta"][:, t] *= live(slope[:, t])
        g["delta_bias"] += g["delta"][:, t].sum(0)
        dS = np.where(on[..., None], dS * np.exp(dt[:, t, :, None] * A), dS)
    return dict(g, S0=dS, out=out, S=S)
