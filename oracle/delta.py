"""fp64 oracle of the gated delta rule and of the norm with gate -- TEST INFRASTRUCTURE.

numpy, token by token in the order of the definition, sharing no code with the
library:

    e_t = v_t - a_t S_{t-1}^T k_t,  S_t = a_t S_{t-1} + beta_t k_t e_t^T,
    o_t = scale S_t^T q_t,          a_t = exp(log_alpha_t)

with q_t, k_t the rows of key head h / (H / Hk), L2-normalised on request.  The
gradient is the reverse recurrence of these lines.  ``plant`` names one
deliberate mistake, for the tests that prove the pins catch it.
"""
from __future__ import annotations

import numpy as np

EPS_L2 = 1e-6


def _bf16(x):
    """The nearest numbers of eight bits."""
    m, e = np.frexp(x)
    return np.ldexp(np.rint(m * 256), e - 8)


def _rows(x, H, l2):
    """Per value head, and the lengths divided by."""
    x = np.repeat(np.asarray(x, np.float64), H // x.shape[1], axis=1)
    n = np.sqrt((x * x).sum(-1, keepdims=True) + EPS_L2) if l2 else np.ones(x.shape[:-1] + (1,))
    return x / n, n


def _start(S0, v, d):
    B, H, _, dv = v.shape
    return np.zeros((B, H, d, dv)) if S0 is None else np.array(S0, np.float64)


def _decays(log_alpha, beta):
    return np.ones_like(beta) if log_alpha is None else np.exp(np.asarray(log_alpha, np.float64))


def _token(S, k, v, b, a, plant=None):
    if plant == "bf16_state":
        S = _bf16(S)
    Sd = S * a[..., None, None]
    seen = S if plant == "undecayed_error" else Sd
    e = v - np.einsum("bhij,bhi->bhj", seen, k)
    if plant == "additive":
        e = v
    return Sd, e, Sd + np.einsum("bhi,bhj->bhij", k, b[..., None] * e)


def forward(q, k, v, beta, log_alpha=None, *, scale, l2=True, S0=None, plant=None, magnitude=False):
    """(out, S) [B,H,N,dv], [B,H,d,dv]; with magnitude also, per output, the
    sum of the absolute terms that any order of the computation adds up."""
    v, beta = np.asarray(v, np.float64), np.asarray(beta, np.float64)
    H = v.shape[1]
    q, k = _rows(q, H, l2)[0] * scale, _rows(k, H, l2)[0]
    a = _decays(log_alpha, beta)
    S = _start(S0, v, k.shape[-1])
    out, mag, Sm = np.empty_like(v), np.empty_like(v), np.abs(S)
    for t in range(v.shape[2]):
        before = S
        _, e, S = _token(S, k[:, :, t], v[:, :, t], beta[:, :, t], a[:, :, t], plant)
        read = before if plant == "read_before_write" else _bf16(S) if plant == "bf16_read" else S
        out[:, :, t] = np.einsum("bhij,bhi->bhj", read, q[:, :, t])
        if magnitude:
            u = np.abs(beta[:, :, t, None] * e)
            Sm = Sm * a[:, :, t, None, None] + np.einsum("bhi,bhj->bhij", np.abs(k[:, :, t]), u)
            mag[:, :, t] = np.einsum("bhij,bhi->bhj", Sm, np.abs(q[:, :, t]))
    return (out, S, mag) if magnitude else (out, S)


def backward(dout, q, k, v, beta, log_alpha=None, *, scale, l2=True, S0=None, dS_out=None,
             plant=None):
    """dq, dk, dv, dbeta, dlog_alpha, dS0."""
    v, beta = np.asarray(v, np.float64), np.asarray(beta, np.float64)
    dout = np.asarray(dout, np.float64)
    B, H, N, _ = v.shape
    Hk, d = k.shape[1], k.shape[-1]
    (q, nq), (k, nk) = _rows(q, H, l2), _rows(k, H, l2)
    a = _decays(log_alpha, beta)
    S = _start(S0, v, d)
    kept = []
    for t in range(N):
        Sd, e, S = _token(S, k[:, :, t], v[:, :, t], beta[:, :, t], a[:, :, t],
                          plant if plant == "bf16_state" else None)
        kept.append((Sd, e, S))
    dS = np.zeros((B, H, d, v.shape[-1])) if dS_out is None else np.array(dS_out, np.float64)
    dq, dk, dv, db, dg = (np.zeros_like(x) for x in (q, k, v, beta, beta))
    for t in reversed(range(N)):
        Sd, e, St = kept[t]
        b = beta[:, :, t, None]
        do, kt = dout[:, :, t], k[:, :, t]
        dq[:, :, t] = scale * np.einsum("bhij,bhj->bhi", _bf16(St) if plant == "bf16_read" else St, do)
        dS = dS + scale * np.einsum("bhi,bhj->bhij", q[:, :, t], do)
        du = np.einsum("bhij,bhi->bhj", dS, kt)
        dv[:, :, t] = b * du
        db[:, :, t] = (du * e).sum(-1)
        dk[:, :, t] = np.einsum("bhij,bhj->bhi", dS, _bf16(b * e) if plant == "bf16_written" else b * e)
        if plant != "key_only_written":
            dk[:, :, t] -= np.einsum("bhij,bhj->bhi", Sd, b * du)
        dS = dS - np.einsum("bhi,bhj->bhij", kt, b * du)
        dg[:, :, t] = (dS * Sd).sum((-1, -2))
        dS = dS * a[:, :, t, None, None]

    def heads(g, unit, length):
        if l2 and plant != "norm_not_differentiated":
            g = g - unit * (unit * g).sum(-1, keepdims=True)
        return (g / length).reshape(B, Hk, H // Hk, N, d).sum(2)

    return heads(dq, q, nq), heads(dk, k, nk), dv, db, dg, dS


def _act(g, activation):
    if activation == "none":
        return g, np.ones_like(g)
    s = 1.0 / (1.0 + np.exp(-g))
    return (s, s * (1 - s)) if activation == "sigmoid" else (g * s, s + g * s * (1 - s))


def norm_gate(x, gate=None, weight=None, *, activation="silu", eps=1e-6, dy=None):
    """y, or (y, dx, dgate, dweight) for dy; x [B,H,N,dv], gate, y, dy [B,N,H,dv]."""
    x = np.moveaxis(np.asarray(x, np.float64), 1, 2)
    w = 1.0 if weight is None else np.asarray(weight, np.float64)
    a, slope = (1.0, 0.0) if gate is None else _act(np.asarray(gate, np.float64), activation)
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    xh = x * r
    y = xh * w * a
    if dy is None:
        return y
    dy = np.asarray(dy, np.float64)
    c = dy * w * a
    dx = r * (c - xh * (c * xh).mean(-1, keepdims=True))
    dw = (dy * xh * a).sum((0, 1))
    if weight is not None and np.ndim(weight) == 1:
        dw = dw.sum(0)
    return y, np.moveaxis(dx, 2, 1), dy * w * xh * slope, dw
