"""What the gated delta rule and the norm with gate behind it are measured on.

Operators (``own`` False: elementary torch operations; ``own`` True: the
library's entry points):

  forward     la_forward_delta       chunked prefill / training forward
  decode      la_decode_step_delta   one token per sequence on a stored state
  backward    la_backward_delta      gradients of the forward
  norm        la_norm_gate           per-head RMS norm, weight and gate
  norm_grad   la_norm_gate and la_norm_gate_backward, a training step's pair

The recurrence per value head (a_t = exp(log_alpha_t), rows of q and k
optionally L2-normalised, value head h reading key head h * Hk / H):

  e_t = v_t - a_t S_{t-1}^T k_t,   S_t = a_t S_{t-1} + beta_t k_t e_t^T,
  o_t = scale S_t^T q_t
"""
import math

import torch

own = False

EPS_L2 = 1e-6    # x / sqrt(|x|^2 + EPS_L2)
EPS_RMS = 1e-6
CHUNK = 64       # tokens per chunk of the plain form
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def _delta(name, op, B, H, Hk, N, d, dv, dtype="bf16", l2=True, gated=True, state=False):
    return {"name": name, "op": op, "B": B, "H": H, "Hk": Hk, "N": N, "d": d, "dv": dv,
            "dtype": dtype, "l2": l2, "gated": gated, "state": state}


def _norm(name, op, B, H, N, dv, x="bf16", dtype="bf16", act="silu", weight="shared"):
    return {"name": name, "op": op, "B": B, "H": H, "N": N, "dv": dv, "x": x, "dtype": dtype,
            "act": act, "weight": weight}


def listed():
    return [
        # a layer's prefill at the library's RetNet / GLA benchmark shape, the state handed to decode
        _delta("fwd_b4_h8_n8192_d128", "forward", 4, 8, 8, 8192, 128, 128, state=True),
        # training forward over many heads, keys shared by two value heads, a ragged length
        _delta("fwd_b16_h32_n2011_d128", "forward", 16, 32, 16, 2011, 128, 128),
        # a short ragged fp32 sequence continued from a state: no gate, keys as given
        _delta("fwd_b2_h4_n333_fp32", "forward", 2, 4, 4, 333, 64, 128, dtype="fp32", l2=False,
               gated=False, state=True),
        # serving: the library's batched-decode workload
        _delta("decode_b256_h32_d128", "decode", 256, 32, 32, 1, 128, 128, state=True),
        # serving: an odd batch with shared keys and smaller heads
        _delta("decode_b37_h12_d64", "decode", 37, 12, 6, 1, 64, 128, state=True),
        # one sequence, one token, fp32: latency
        _delta("decode_b1_h8_fp32", "decode", 1, 8, 8, 1, 64, 64, dtype="fp32", state=True),
        # training step of one layer at the benchmark shape
        _delta("bwd_b4_h8_n8192_d128", "backward", 4, 8, 8, 8192, 128, 128),
        # many heads, shared keys, ragged, with a gradient of the final state
        _delta("bwd_b8_h32_n1037_d128", "backward", 8, 32, 8, 1037, 128, 128, state=True),
        # a short fp32 training sequence, no gate
        _delta("bwd_b2_h4_n201_fp32", "backward", 2, 4, 2, 201, 64, 64, dtype="fp32", gated=False),
        # norm and gate behind the headline forward (fp32 outputs, d = 64)
        _norm("norm_b2_h16_n32768_d64", "norm", 2, 16, 32768, 64, x="fp32"),
        # training pair at the layer's shape
        _norm("norm_grad_b4_h8_n8192_d128", "norm_grad", 4, 8, 8192, 128),
        # a short ragged pair in fp32 with a weight for each head
        _norm("norm_grad_b3_h6_n1009_fp32", "norm_grad", 3, 6, 1009, 64, x="fp32", dtype="fp32",
              act="sigmoid", weight="head"),
    ]


def _spread(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["forward", "decode", "backward", "norm", "norm_grad"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    if op in ("norm", "norm_grad"):
        N = _spread(rng, 1, 32768)
        rows = _spread(rng, 1, max(1, min(512, (1 << 17) // N)))
        H = rng.randint(1, min(rows, 16))
        return {"op": op, "B": max(1, rows // H), "H": H, "N": N, "dv": rng.choice([32, 64, 128]),
                "x": rng.choice([dtype, "fp32"]), "dtype": dtype,
                "act": rng.choice(["silu", "sigmoid"]), "weight": rng.choice(["shared", "head"])}
    Hk = rng.choice([1, 2, 3, 4, 8])
    H = Hk * rng.choice([1, 1, 2, 4])
    d, dv = rng.choice([32, 64, 128, 128]), rng.choice([32, 64, 128, 128])
    if op == "decode":
        B, N = _spread(rng, 1, 8192 // H), 1
    else:
        N = _spread(rng, 1, 32768 if op == "forward" else 8192)
        most = 1_000_000 if op == "forward" else 250_000
        if dtype == "fp32":
            most //= 8
        N = min(N, most // H)
        B = _spread(rng, 1, max(1, min(64, most // (H * N))))
    return {"op": op, "B": B, "H": H, "Hk": Hk, "N": N, "d": d, "dv": dv, "dtype": dtype,
            "l2": rng.random() < 0.7, "gated": rng.random() < 0.8,
            "state": op == "decode" or rng.random() < 0.5}


def _randn(gen, shape, dtype, scale=1.0):
    x = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)
    return (x * scale).to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    s = {"case": case}
    B, H, N, dv = case["B"], case["H"], case["N"], case["dv"]
    dtype = DTYPES[case["dtype"]]
    if case["op"] in ("norm", "norm_grad"):
        s["x"] = _randn(gen, (B, H, N, dv), DTYPES[case["x"]])
        s["gate"] = _randn(gen, (B, N, H, dv), dtype)
        shape = (dv,) if case["weight"] == "shared" else (H, dv)
        s["weight"] = 1.0 + _randn(gen, shape, torch.float32, 0.1)
        if case["op"] == "norm_grad":
            s["dy"] = _randn(gen, (B, N, H, dv), dtype)
        return s
    Hk, d = case["Hk"], case["d"]
    # keys of about unit length: normalised inside, or scaled as the projections of a layer leave them
    qk_scale = 1.0 if case["l2"] else d ** -0.5
    tok = (N,) if case["op"] != "decode" else ()
    s["q"] = _randn(gen, (B, Hk) + tok + (d,), dtype, qk_scale)
    s["k"] = _randn(gen, (B, Hk) + tok + (d,), dtype, qk_scale)
    s["v"] = _randn(gen, (B, H) + tok + (dv,), dtype)
    s["beta"] = torch.sigmoid(_randn(gen, (B, H) + tok, torch.float32))
    s["log_alpha"] = None
    if case["gated"]:
        # -A softplus(x + bias): rates A in [1, 16] and steps in [1e-3, 1e-1] per head
        u = torch.rand((2, H), generator=gen, device="cuda", dtype=torch.float32)
        rate = 1.0 + 15.0 * u[0]
        step = torch.exp(math.log(1e-3) + u[1] * math.log(100.0))
        bias = step + torch.log(-torch.expm1(-step))
        x = _randn(gen, (B, H) + tok, torch.float32)
        one = (1, H) + (1,) * len(tok)
        s["log_alpha"] = -rate.view(one) * torch.nn.functional.softplus(x + bias.view(one))
    if case["state"]:
        s["S0"] = _randn(gen, (B, H, d, dv), torch.float32, 0.3)
    if case["op"] == "backward":
        s["dout"] = _randn(gen, (B, H, N, dv), dtype)
        if case["state"]:
            s["dS"] = _randn(gen, (B, H, d, dv), torch.float32, 0.3)
    return s


# ---- the plain form --------------------------------------------------------

def _unit(x):
    return x * torch.rsqrt((x * x).sum(-1, keepdim=True) + EPS_L2)


def _solve_lower(A):
    """(I + A)^{-1} of strictly lower A [..., n, n], n a power of two: blocks of 1, 2, 4, ... joined."""
    n = A.shape[-1]
    T = torch.ones(A.shape[:-2] + (n, 1, 1), dtype=A.dtype, device=A.device)
    size = 1
    while size < n:
        pairs = n // (2 * size)
        blocks = A.reshape(A.shape[:-2] + (pairs, 2 * size, pairs, 2 * size))
        at = torch.arange(pairs, device=A.device)
        low = blocks[..., at, :, at, :].movedim(0, -3)[..., size:, :size]
        upper, lower = T[..., 0::2, :, :], T[..., 1::2, :, :]
        corner = -(lower @ low @ upper)
        T = torch.cat([torch.cat([upper, torch.zeros_like(upper)], -1),
                       torch.cat([corner, lower], -1)], -2)
        size *= 2
    return T[..., 0, :, :]


def _plain_forward(q, k, v, beta, log_alpha, S, scale, l2):
    """Chunked over CHUNK tokens, in 32 bits (the gates' running sums in 64)."""
    B, H, N, dv = v.shape
    groups = H // k.shape[1]
    if l2:
        q, k = _unit(q), _unit(k)
    q = (q * scale).repeat_interleave(groups, 1)
    k = k.repeat_interleave(groups, 1)
    pad = -N % CHUNK
    n = (N + pad) // CHUNK

    def chunks(x):
        x = torch.cat([x, x.new_zeros(x.shape[:2] + (pad,) + x.shape[3:])], 2) if pad else x
        return x.reshape(x.shape[:2] + (n, CHUNK) + x.shape[3:])

    q, k, v, beta = chunks(q), chunks(k), chunks(v), chunks(beta)
    lower = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=v.device).tril()
    if log_alpha is None:
        decay = lower.to(v.dtype)
        from_start = torch.ones_like(beta)
        to_end = from_start
    else:
        G = chunks(log_alpha).double().cumsum(-1)
        diff = (G[..., :, None] - G[..., None, :]).masked_fill(~lower, -math.inf)
        decay = diff.exp().to(v.dtype)
        from_start = G.exp().to(v.dtype)
        to_end = (G[..., -1:] - G).exp().to(v.dtype)
    A = ((k * beta[..., None]) @ k.transpose(-1, -2) * decay).tril(-1)
    T = _solve_lower(A) * beta[..., None, :]
    W = T @ (k * from_start[..., None])
    TV = T @ v
    P = q @ k.transpose(-1, -2) * decay
    q_in = q * from_start[..., None]
    k_out = (k * to_end[..., None]).transpose(-1, -2)
    outs = []
    for c in range(n):
        U = TV[:, :, c] - W[:, :, c] @ S
        outs.append(q_in[:, :, c] @ S + P[:, :, c] @ U)
        S = S * from_start[:, :, c, -1, None, None] + k_out[:, :, c] @ U
    out = torch.stack(outs, 2).reshape(B, H, n * CHUNK, dv)[:, :, :N]
    return out, S


def _plain_delta(s):
    c = s["case"]
    scale = c["d"] ** -0.5
    back = c["op"] == "backward"
    q, k, v, beta = (s[n].float().requires_grad_(back) if back else s[n].float()
                     for n in ("q", "k", "v", "beta"))
    log_alpha = s["log_alpha"]
    if back:
        beta = s["beta"].clone().requires_grad_()
        q, k, v = (s[n].float().clone().requires_grad_() for n in ("q", "k", "v"))
        log_alpha = log_alpha.clone().requires_grad_() if log_alpha is not None else None
    if c["state"]:
        S = s["S0"].clone().requires_grad_() if back else s["S0"]
    else:
        S = torch.zeros(c["B"], c["H"], c["d"], c["dv"], device="cuda")
    S_in = S
    out, S_last = _plain_forward(q, k, v, beta, log_alpha, S, scale, c["l2"])
    if not back:
        r = {"out": out.to(DTYPES[c["dtype"]])}
        if c["state"]:
            r["S"] = S_last
        return r
    wanted = {"dq": q, "dk": k, "dv": v, "dbeta": beta}
    if log_alpha is not None:
        wanted["dlog_alpha"] = log_alpha
    if c["state"]:
        wanted["dS0"] = S_in
    loss = [out] + ([S_last] if c["state"] else [])
    grads = torch.autograd.grad(loss, list(wanted.values()),
                                [s["dout"].float()] + ([s["dS"]] if c["state"] else []))
    r = dict(zip(wanted, grads))
    for n in ("dq", "dk", "dv"):
        r[n] = r[n].to(DTYPES[c["dtype"]])
    return r


def _plain_decode(s):
    c = s["case"]
    groups = c["H"] // c["Hk"]
    q, k, v = s["q"].float(), s["k"].float(), s["v"].float()
    if c["l2"]:
        q, k = _unit(q), _unit(k)
    q = (q * c["d"] ** -0.5).repeat_interleave(groups, 1)
    k = k.repeat_interleave(groups, 1)
    S = s["S0"]
    if s["log_alpha"] is not None:
        S = S * s["log_alpha"].exp()[..., None, None]
    e = v - (k[..., None, :] @ S)[..., 0, :]
    S = S + k[..., :, None] * (s["beta"][..., None] * e)[..., None, :]
    out = (q[..., None, :] @ S)[..., 0, :]
    s["S0"].copy_(S)
    return {"out": out.to(DTYPES[c["dtype"]]), "S": s["S0"]}


def _plain_norm(s):
    c = s["case"]
    dtype = DTYPES[c["dtype"]]
    x = s["x"].float().transpose(1, 2)
    g, w = s["gate"].float(), s["weight"]
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS_RMS)
    xh = x * r
    sig = torch.sigmoid(g)
    act = g * sig if c["act"] == "silu" else sig
    y = (w * xh * act).to(dtype)
    if c["op"] == "norm":
        return {"y": y}
    dact = sig * (1.0 + g * (1.0 - sig)) if c["act"] == "silu" else sig * (1.0 - sig)
    dy = s["dy"].float()
    t = dy * w * act
    dx = r * (t - xh * (t * xh).mean(-1, keepdim=True))
    axes = (0, 1, 2) if c["weight"] == "shared" else (0, 1)
    dw = (dy * xh * act).sum(axes, dtype=torch.float64).float()
    return {"y": y, "dx": dx.transpose(1, 2).contiguous().to(s["x"].dtype),
            "dgate": (dy * w * xh * dact).to(dtype), "dweight": dw}


# ---- the library's calls ---------------------------------------------------

def _own_run(s):
    import kernelised_causal_linear_gb300 as la

    c = s["case"]
    if c["op"] in ("norm", "norm_grad"):
        y = la.la_norm_gate(s["x"], s["gate"], s["weight"], activation=c["act"], eps=EPS_RMS)
        if c["op"] == "norm":
            return {"y": y}
        dx, dgate, dw = la.la_norm_gate_backward(s["dy"], s["x"], s["gate"], s["weight"],
                                                 activation=c["act"], eps=EPS_RMS)
        return {"y": y, "dx": dx, "dgate": dgate, "dweight": dw}
    fm = "l2" if c["l2"] else "none"
    if c["op"] == "decode":
        out = la.la_decode_step_delta(s["S0"], s["q"], s["k"], s["v"], s["beta"], s["log_alpha"],
                                      feature_map=fm)
        return {"out": out, "S": s["S0"]}
    if c["op"] == "forward":
        out, S = la.la_forward_delta(s["q"], s["k"], s["v"], s["beta"], s["log_alpha"],
                                     feature_map=fm, S0=s.get("S0"), return_state=c["state"])
        return {"out": out, "S": S} if c["state"] else {"out": out}
    dq, dk, dv, dbeta, dlog_alpha, dS0 = la.la_backward_delta(
        s["dout"], s["q"], s["k"], s["v"], s["beta"], s["log_alpha"], feature_map=fm,
        S0=s.get("S0"), dS_out=s.get("dS"))
    r = {"dq": dq, "dk": dk, "dv": dv, "dbeta": dbeta}
    if dlog_alpha is not None:
        r["dlog_alpha"] = dlog_alpha
    if dS0 is not None:
        r["dS0"] = dS0
    return r


def run(state):
    if own:
        return _own_run(state)
    op = state["case"]["op"]
    if op in ("norm", "norm_grad"):
        return _plain_norm(state)
    return _plain_decode(state) if op == "decode" else _plain_delta(state)


def work(case):
    """Each input read once, each output written once; the recurrence's own products."""
    B, H, N, dv = case["B"], case["H"], case["N"], case["dv"]
    es = 2 if case["dtype"] == "bf16" else 4
    if case["op"] in ("norm", "norm_grad"):
        n = B * H * N * dv
        xs = 2 if case["x"] == "bf16" else 4
        if case["op"] == "norm":
            return {"bytes": n * (xs + 2 * es), "flops": 12 * n}
        # the pair: y from x, gate; then dx, dgate, dweight from dy, x, gate
        return {"bytes": n * (xs + 2 * es) + n * (2 * xs + 3 * es), "flops": 40 * n}
    Hk, d = case["Hk"], case["d"]
    qk, vo = B * Hk * N * d * es, B * H * N * dv * es
    gates = B * H * N * 4 * (2 if case["gated"] else 1)
    state = B * H * d * dv * 4
    steps = B * H * N * d * dv
    if case["op"] == "backward":
        return {"bytes": 4 * qk + 3 * vo + 2 * gates + (3 * state if case["state"] else 0),
                "flops": 18 * steps}
    return {"bytes": 2 * qk + 2 * vo + gates + (2 * state if case["state"] else 0),
            "flops": 6 * steps}


# ---- 64 bits, token by token -----------------------------------------------

def _exact_tokens(s):
    """Inputs in 64 bits, [token][B,H,...], q and k per value head before scale and norm."""
    c = s["case"]
    one = c["op"] == "decode"

    def tok(x):
        x = x.double()
        return x[None] if one else x.movedim(2, 0)

    at = torch.arange(c["H"], device="cuda") * c["Hk"] // c["H"]
    q, k = tok(s["q"]).index_select(2, at), tok(s["k"]).index_select(2, at)
    a = torch.exp(tok(s["log_alpha"])) if s["log_alpha"] is not None else None
    S = s["S0"].double() if c["state"] else torch.zeros(
        c["B"], c["H"], c["d"], c["dv"], dtype=torch.float64, device="cuda")
    return q, k, tok(s["v"]), tok(s["beta"]), a, S


def _lengths(x, l2):
    return torch.sqrt((x ** 2).sum(-1, keepdim=True) + EPS_L2) if l2 else torch.ones_like(x[..., :1])


def _step(S, k, v, beta, a):
    S = S if a is None else S * a[..., None, None]
    e = v - torch.einsum("bhij,bhi->bhj", S, k)
    return S, e, S + torch.einsum("bhi,bhj->bhij", k, beta[..., None] * e)


def _exact_forward(s):
    c = s["case"]
    q, k, v, beta, a, S = _exact_tokens(s)
    q = q / _lengths(q, c["l2"]) / math.sqrt(c["d"])
    k = k / _lengths(k, c["l2"])
    out = torch.empty_like(v)
    for t in range(q.shape[0]):
        _, _, S = _step(S, k[t], v[t], beta[t], None if a is None else a[t])
        out[t] = torch.einsum("bhij,bhi->bhj", S, q[t])
    if c["op"] == "decode":
        return {"out": out[0], "S": S}
    return {"out": out.movedim(0, 2), "S": S} if c["state"] else {"out": out.movedim(0, 2)}


def _exact_backward(s):
    c = s["case"]
    q, k, v, beta, a, S = _exact_tokens(s)
    lq, lk = _lengths(q, c["l2"]), _lengths(k, c["l2"])
    q, k = q / lq, k / lk
    dout = s["dout"].double().movedim(2, 0) / math.sqrt(c["d"])
    N, every = q.shape[0], 64
    starts = []
    for t in range(N):
        if t % every == 0:
            starts.append(S)
        _, _, S = _step(S, k[t], v[t], beta[t], None if a is None else a[t])
    dS = s["dS"].double() if c["state"] else torch.zeros_like(S)
    dq, dk, dv, dbeta = (torch.empty_like(x) for x in (q, k, v, beta))
    dg = torch.empty_like(beta)
    for b in reversed(range(len(starts))):
        lo, hi = b * every, min(N, (b + 1) * every)
        kept, S = [], starts[b]
        for t in range(lo, hi):
            Sd, e, S = _step(S, k[t], v[t], beta[t], None if a is None else a[t])
            kept.append((Sd, e, S))
        for t in reversed(range(lo, hi)):
            Sd, e, St = kept[t - lo]
            bt = beta[t][..., None]
            dq[t] = torch.einsum("bhij,bhj->bhi", St, dout[t])
            dS = dS + torch.einsum("bhi,bhj->bhij", q[t], dout[t])
            du = torch.einsum("bhij,bhi->bhj", dS, k[t])
            dv[t] = bt * du
            dbeta[t] = (du * e).sum(-1)
            dk[t] = torch.einsum("bhij,bhj->bhi", dS, bt * e) - torch.einsum("bhij,bhj->bhi", Sd, bt * du)
            dS = dS - torch.einsum("bhi,bhj->bhij", k[t], bt * du)
            dg[t] = (dS * Sd).sum((-1, -2))
            if a is not None:
                dS = dS * a[t][..., None, None]

    def heads(x, unit, length):  # back through the length, then over the value heads of a key head
        if c["l2"]:
            x = (x - unit * (unit * x).sum(-1, keepdim=True)) / length
        return x.movedim(0, 2).reshape(c["B"], c["Hk"], c["H"] // c["Hk"], N, c["d"]).sum(2)

    r = {"dq": heads(dq, q, lq), "dk": heads(dk, k, lk), "dv": dv.movedim(0, 2),
         "dbeta": dbeta.movedim(0, 2)}
    if a is not None:
        r["dlog_alpha"] = dg.movedim(0, 2)
    if c["state"]:
        r["dS0"] = dS
    return r


def _exact_norm(s):
    c = s["case"]
    x, g, w = s["x"].double().movedim(1, 2), s["gate"].double(), s["weight"].double()
    length = torch.sqrt((x ** 2).sum(-1, keepdim=True) / c["dv"] + EPS_RMS)
    unit = x / length
    sig = 1.0 / (1.0 + torch.exp(-g))
    silu = c["act"] == "silu"
    act = sig * g if silu else sig
    r = {"y": unit * w * act}
    if c["op"] == "norm":
        return r
    slope = sig * (1.0 - sig)
    dy = s["dy"].double()
    inner = dy * act * w
    r["dx"] = ((inner - unit * (unit * inner).sum(-1, keepdim=True) / c["dv"]) / length).movedim(2, 1)
    r["dgate"] = dy * unit * w * (sig + g * slope if silu else slope)
    dw = (dy * unit * act).sum((0, 1))
    r["dweight"] = dw.sum(0) if c["weight"] == "shared" else dw
    return r


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("norm", "norm_grad"):
        return _exact_norm(s)
    return _exact_backward(s) if case["op"] == "backward" else _exact_forward(s)
