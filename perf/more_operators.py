"""What the selective state-space scan and the short causal convolution in front of
it are measured on.

Operators (``own`` False: elementary torch operations; ``own`` True: the
library's entry points):

  conv       la_forward_conv        short causal convolution, prefill and training
  conv_step  la_decode_step_conv    one token per sequence on a stored window
  conv_grad  la_backward_conv       gradients of the convolution
  ssm        la_forward_ssm         selective scan, prefill and training
  ssm_step   la_decode_step_ssm     one token per sequence on a stored state
  ssm_grad   la_backward_ssm        gradients of the scan

The convolution, per channel c with W taps (x before the first token from the
window S, oldest row first):

  y_t = act(bias + sum_j w[c,j] x_{t-W+1+j})

The scan, per channel c and state s, with dt_t = softplus(delta_t + delta_bias)
and B, C shared by the channels of a group:

  S_t = exp(dt_t A) S_{t-1} + dt_t x_t B_t,   y_t = sum_s C_t S_t + D x_t
  out_t = y_t silu(z_t)

With lengths, row b stops after lengths[b] tokens: its state is the one there,
outputs and gradients behind it are zero.
"""
import math

import torch

own = False

CHUNK = 64  # tokens per chunk of the plain form
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def _conv(name, op, B, N, C, W=4, heads=0, dtype="bf16", act="silu", state=False, ragged=False, slices=False):
    return {"name": name, "op": op, "B": B, "N": N, "C": C, "W": W, "heads": heads, "dtype": dtype,
            "act": act, "state": state, "ragged": ragged, "slices": slices}


def _ssm(name, op, B, N, C, n=16, G=1, dtype="bf16", gate=True, state=False, ragged=False, slices=False):
    return {"name": name, "op": op, "B": B, "N": N, "C": C, "n": n, "G": G, "dtype": dtype, "gate": gate,
            "state": state, "ragged": ragged, "slices": slices}


def listed():
    return [
        # queries, keys and values of 32 heads of 128 in front of a layer's prefill, one wide slice of
        # a projection, head-major for the attention calls
        _conv("conv_b4_n8192_c4096_heads", "conv", 4, 8192, 4096, heads=32, slices=True),
        # a short ragged fp32 batch continued from windows, an odd number of channels
        _conv("conv_b3_n333_c197_fp32", "conv", 3, 333, 197, W=3, dtype="fp32", state=True, ragged=True),
        # serving: the library's batched-decode workload, 32 heads of 128
        _conv("conv_step_b256_c4096", "conv_step", 256, 1, 4096, state=True),
        # one sequence, one token, fp32: latency
        _conv("conv_step_b1_c512_fp32", "conv_step", 1, 1, 512, dtype="fp32", state=True),
        # training step of one layer
        _conv("conv_grad_b4_n8192_c2048", "conv_grad", 4, 8192, 2048, slices=True),
        # a short ragged training batch from head-major gradients
        _conv("conv_grad_b8_n1037_c768", "conv_grad", 8, 1037, 768, heads=12, state=True, ragged=True),
        # a layer's prefill at the library's RetNet / GLA benchmark length, the state handed to decode
        _ssm("ssm_b4_n8192_c2048", "ssm", 4, 8192, 2048, state=True, slices=True),
        # a short ragged fp32 batch, an odd number of channels, no gate
        _ssm("ssm_b2_n333_c197_fp32", "ssm", 2, 333, 197, dtype="fp32", gate=False, state=True, ragged=True),
        # serving: the batched-decode workload's batch
        _ssm("ssm_step_b256_c4096", "ssm_step", 256, 1, 4096, state=True, slices=True),
        # an odd batch with two groups and more states, fp32: latency
        _ssm("ssm_step_b5_c250_n32_fp32", "ssm_step", 5, 1, 250, n=32, G=2, dtype="fp32", state=True),
        # training step of one layer
        _ssm("ssm_grad_b4_n2048_c2048", "ssm_grad", 4, 2048, 2048, slices=True),
        # a ragged fp32 training batch with groups and gradients of the final state
        _ssm("ssm_grad_b3_n701_c600_fp32", "ssm_grad", 3, 701, 600, G=3, dtype="fp32", state=True, ragged=True),
    ]


def _spread(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["conv", "conv_step", "conv_grad", "ssm", "ssm_step", "ssm_grad"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    step = op.endswith("step")
    most = {"conv": 8192 * 4096 * 4, "conv_step": 256 * 4096, "conv_grad": 8192 * 2048 * 4,
            "ssm": 8192 * 2048 * 4, "ssm_step": 256 * 4096, "ssm_grad": 2048 * 2048 * 4}[op]
    if dtype == "fp32":
        most //= 4
    N = 1 if step else _spread(rng, 1, 8192 if op == "ssm_grad" else 32768)
    C = _spread(rng, 32, min(4096, most // N))
    if rng.random() < 0.6:  # widths are most often round
        C = max(32, C // 32 * 32)
    c = {"op": op, "N": N, "C": C, "dtype": dtype, "state": step or rng.random() < 0.5,
         "ragged": not step and rng.random() < 0.3, "slices": rng.random() < 0.5}
    if op.startswith("conv"):
        c["W"] = rng.choice([2, 3, 4, 4])
        c["act"] = rng.choice(["silu", "silu", "none"])
        c["heads"] = C // 32 if not step and C % 32 == 0 and rng.random() < 0.5 else 0
    else:
        c["n"] = rng.choice([8, 16, 16, 32, 64])
        most = most * 16 // c["n"]
        c["G"] = 2 if C % 2 == 0 and rng.random() < 0.25 else 1
        c["gate"] = rng.random() < 0.8
    c["B"] = _spread(rng, 1, max(1, min(256 if step else 64, most // (N * C))))
    return c


def _randn(gen, shape, dtype, scale=1.0):
    x = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)
    return (x * scale).to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    c, dtype, f32 = case, DTYPES[case["dtype"]], torch.float32
    B, N, C = c["B"], c["N"], c["C"]
    tok = () if c["op"].endswith("step") else (N,)
    s = {"case": c, "lengths": None}
    if c["ragged"]:
        s["lengths"] = torch.randint(0, N + 1, (B,), generator=gen, device="cuda", dtype=torch.int32)

    def pair(width):
        """Two inputs side by side in one projection's rows, or apart."""
        if c["slices"]:
            both = _randn(gen, (B,) + tok + (2 * width,), dtype)
            return both[..., :width], both[..., width:]
        return _randn(gen, (B,) + tok + (width,), dtype), _randn(gen, (B,) + tok + (width,), dtype)

    if c["op"].startswith("conv"):
        s["x"] = pair(C)[0]
        s["weight"] = _randn(gen, (C, c["W"]), f32, c["W"] ** -0.5)
        s["bias"] = _randn(gen, (C,), f32, 0.1)
        if c["state"]:
            s["S0"] = _randn(gen, (B, c["W"] - 1, C), dtype)
        if c["op"] == "conv_grad":
            s["dy"] = _randn(gen, (B, c["heads"], N, C // c["heads"]) if c["heads"] else (B, N, C), dtype)
            if c["state"]:
                s["dS"] = _randn(gen, (B, c["W"] - 1, C), dtype)
        return s
    n, G = c["n"], c["G"]
    s["x"], s["z"] = pair(C)
    if not c["gate"]:
        s["z"] = None
    s["delta"] = _randn(gen, (B,) + tok + (C,), dtype, 0.5)
    if c["slices"]:  # B and C behind the low-rank step's own columns
        rank = max(1, C // 32)
        rows = _randn(gen, (B,) + tok + (rank + 2 * G * n,), dtype)
        s["Bm"] = rows[..., rank:rank + G * n].unflatten(-1, (G, n))
        s["Cm"] = rows[..., rank + G * n:].unflatten(-1, (G, n))
    else:
        s["Bm"] = _randn(gen, (B,) + tok + (G, n), dtype)
        s["Cm"] = _randn(gen, (B,) + tok + (G, n), dtype)
    # rates near 1 .. n, steps of 1e-3 to 1e-1
    s["A"] = -torch.exp(torch.log(torch.arange(1, n + 1, device="cuda", dtype=f32)) + _randn(gen, (C, n), f32, 0.2))
    step = torch.exp(math.log(1e-3) + math.log(100.0) * torch.rand((C,), generator=gen, device="cuda"))
    s["delta_bias"] = step + torch.log(-torch.expm1(-step))
    s["D"] = 1.0 + _randn(gen, (C,), f32, 0.1)
    if c["state"]:
        s["S0"] = _randn(gen, (B, C, n), f32, 0.3)
    if c["op"] == "ssm_grad":
        s["dout"] = _randn(gen, (B, N, C), dtype)
        if c["state"]:
            s["dS"] = _randn(gen, (B, C, n), f32, 0.3)
    return s


# ---- the plain form --------------------------------------------------------

def _live(s):
    """[B,N,1] truth of the tokens that a row has."""
    at = torch.arange(s["case"]["N"], device="cuda")
    return (at[None] < s["lengths"][:, None])[..., None]


def _to_heads(y, c):
    return y.unflatten(-1, (c["heads"], -1)).transpose(1, 2) if c["heads"] else y


def _plain_conv_forward(x, w, bias, S0, s):
    """(y [B,N,C], the last W-1 inputs of each row)."""
    c = s["case"]
    N, W = c["N"], c["W"]
    x = torch.cat([S0 if S0 is not None else x.new_zeros(c["B"], W - 1, c["C"]), x], 1)
    u = bias + sum(w[:, j] * x[:, j:j + N] for j in range(W))
    y = u * torch.sigmoid(u) if c["act"] == "silu" else u
    end = torch.full((c["B"],), N, device="cuda") if s["lengths"] is None else s["lengths"].long()
    rows = (end[:, None] + torch.arange(W - 1, device="cuda"))[..., None].expand(-1, -1, c["C"])
    if s["lengths"] is not None:
        y = torch.where(_live(s), y, torch.zeros_like(y))
    return y, x.gather(1, rows)


def _plain_conv(s):
    c, dtype = s["case"], DTYPES[s["case"]["dtype"]]
    S0 = s["S0"].float() if c["state"] else None
    if c["op"] == "conv":
        y, S = _plain_conv_forward(s["x"].float(), s["weight"], s["bias"], S0, s)
        y = _to_heads(y, c).contiguous().to(dtype)
        return {"y": y, "S": S.to(dtype)} if c["state"] else {"y": y}
    leaves = [s["x"].float().clone(), s["weight"].clone(), s["bias"].clone()] + ([S0.clone()] if c["state"] else [])
    leaves = [t.requires_grad_() for t in leaves]
    y, S = _plain_conv_forward(*leaves[:3], leaves[3] if c["state"] else None, s)
    loss, given = [_to_heads(y, c)], [s["dy"].float()]
    if c["state"]:
        loss, given = loss + [S], given + [s["dS"].float()]
    grads = torch.autograd.grad(loss, leaves, given)
    r = {"dx": grads[0].to(dtype), "dweight": grads[1], "dbias": grads[2]}
    if c["state"]:
        r["dS0"] = grads[3].to(dtype)
    return r


def _plain_conv_step(s):
    c, dtype = s["case"], DTYPES[s["case"]["dtype"]]
    rows = torch.cat([s["S0"], s["x"][:, None]], 1)
    u = s["bias"] + (rows.float() * s["weight"].t()).sum(1)
    s["S0"].copy_(rows[:, 1:])
    return {"y": (u * torch.sigmoid(u) if c["act"] == "silu" else u).to(dtype), "S": s["S0"]}


def _softplus(u):
    return u.clamp(min=0) + torch.log1p(torch.exp(-u.abs()))


def _walk(a, b, h, read=None):
    """The recurrence along dimension 2 from h: the last state, and read(t, state) of every token."""
    seen = []
    for t in range(b.shape[2]):
        h = a[:, :, t] * h + b[:, :, t]
        if read is not None:
            seen.append(read(t, h))
    return h, seen


def _plain_ssm_forward(x, delta, A, Bm, Cm, D, z, bias, S0, s):
    """Chunks of CHUNK tokens side by side: their ends from a zero start, the states between them, and
    the run that counts."""
    c = s["case"]
    B, N, C, n, G = c["B"], c["N"], c["C"], c["n"], c["G"]
    dt = _softplus(delta + bias)
    if s["lengths"] is not None:
        live = _live(s)
        zero = torch.zeros((), device="cuda")
        dt, x = torch.where(live, dt, zero), torch.where(live, x, zero)
    pad = -N % CHUNK
    k = (N + pad) // CHUNK

    def chunks(t):
        t = torch.cat([t, t.new_zeros((B, pad) + t.shape[2:])], 1) if pad else t
        return t.reshape((B, k, CHUNK) + t.shape[2:])

    dts, groups = chunks(dt), (B, k, CHUNK, G, C // G, n)
    a = torch.exp(dts[..., None] * A)
    b = ((dts * chunks(x)).unflatten(-1, (G, -1))[..., None] * chunks(Bm)[..., None, :]).reshape(a.shape)
    zero = torch.zeros((B, k, C, n), device="cuda")
    ends, _ = _walk(a, b, zero)
    over = torch.exp(dts.double().sum(2).float()[..., None] * A)
    S = S0 if S0 is not None else zero[:, 0]
    starts = []
    for i in range(k):
        starts.append(S)
        S = over[:, i] * S + ends[:, i]
    c_rows = chunks(Cm)
    _, y = _walk(a, b, torch.stack(starts, 1),
                 lambda t, h: (h.view(B, k, G, C // G, n) * c_rows[:, :, t, :, None]).sum(-1).reshape(B, k, C))
    y = torch.stack(y, 2).reshape(B, k * CHUNK, C)[:, :N] + D * x
    if z is not None:
        y = y * (z * torch.sigmoid(z))
    if s["lengths"] is not None:
        y = torch.where(live, y, zero[0, 0, 0, 0])
    return y, S


SSM_LEAVES = ("x", "delta", "A", "Bm", "Cm", "D", "z", "delta_bias", "S0")


def _plain_ssm(s):
    c, dtype = s["case"], DTYPES[s["case"]["dtype"]]
    ins = [s[n].float() if s.get(n) is not None else None for n in SSM_LEAVES]
    if c["op"] == "ssm":
        out, S = _plain_ssm_forward(*ins, s)
        return {"out": out.to(dtype), "S": S} if c["state"] else {"out": out.to(dtype)}
    ins = [t.clone().requires_grad_() if t is not None else None for t in ins]
    out, S = _plain_ssm_forward(*ins, s)
    wanted = [n for n, t in zip(SSM_LEAVES, ins) if t is not None]
    grads = torch.autograd.grad([out] + ([S] if c["state"] else []), [t for t in ins if t is not None],
                                [s["dout"].float()] + ([s["dS"]] if c["state"] else []))
    return {"d" + n: g.to(s[n].dtype) for n, g in zip(wanted, grads)}


def _plain_ssm_step(s):
    c, dtype = s["case"], DTYPES[s["case"]["dtype"]]
    x, S = s["x"].float(), s["S0"]
    dt = _softplus(s["delta"].float() + s["delta_bias"])
    rows = [s[m].float().repeat_interleave(c["C"] // c["G"], 1) if c["G"] > 1 else s[m].float() for m in ("Bm", "Cm")]
    S = torch.exp(dt[..., None] * s["A"]) * S + (dt * x)[..., None] * rows[0]
    y = (S * rows[1]).sum(-1) + s["D"] * x
    if s["z"] is not None:
        z = s["z"].float()
        y = y * (z * torch.sigmoid(z))
    s["S0"].copy_(S)
    return {"out": y.to(dtype), "S": s["S0"]}


# ---- the library's calls ---------------------------------------------------

def _own_run(s):
    import kernelised_causal_linear_gb300 as la

    c = s["case"]
    if c["op"] == "conv_step":
        y = la.la_decode_step_conv(s["S0"], s["x"], s["weight"], s["bias"], activation=c["act"])
        return {"y": y, "S": s["S0"]}
    if c["op"] == "conv":
        y, S = la.la_forward_conv(s["x"], s["weight"], s["bias"], activation=c["act"], heads=c["heads"] or None,
                                  S0=s.get("S0"), return_state=c["state"], lengths=s["lengths"])
        return {"y": y, "S": S} if c["state"] else {"y": y}
    if c["op"] == "conv_grad":
        dx, dw, db, dS0 = la.la_backward_conv(s["dy"], s["x"], s["weight"], s["bias"], activation=c["act"],
                                              S0=s.get("S0"), dS_out=s.get("dS"), lengths=s["lengths"])
        r = {"dx": dx, "dweight": dw, "dbias": db}
        return dict(r, dS0=dS0) if c["state"] else r
    more = {"D": s["D"], "z": s["z"], "delta_bias": s["delta_bias"], "softplus": True}
    if c["op"] == "ssm_step":
        out = la.la_decode_step_ssm(s["S0"], s["x"], s["delta"], s["A"], s["Bm"], s["Cm"], **more)
        return {"out": out, "S": s["S0"]}
    if c["op"] == "ssm":
        out, S = la.la_forward_ssm(s["x"], s["delta"], s["A"], s["Bm"], s["Cm"], **more, S0=s.get("S0"),
                                   return_state=c["state"], lengths=s["lengths"])
        return {"out": out, "S": S} if c["state"] else {"out": out}
    grads = la.la_backward_ssm(s["dout"], s["x"], s["delta"], s["A"], s["Bm"], s["Cm"], **more, S0=s.get("S0"),
                               dS_out=s.get("dS"), lengths=s["lengths"])
    return {"d" + n: g for n, g in zip(SSM_LEAVES, grads) if s.get(n) is not None}


def run(state):
    if own:
        return _own_run(state)
    op = state["case"]["op"]
    if op.endswith("step"):
        return _plain_conv_step(state) if op == "conv_step" else _plain_ssm_step(state)
    return _plain_conv(state) if op.startswith("conv") else _plain_ssm(state)


def work(case):
    """Each input read once, each output written once; the recurrence's own operations."""
    c = case
    es = 2 if c["dtype"] == "bf16" else 4
    tokens = c["B"] * c["N"]
    rows = tokens * c["C"]
    if c["op"].startswith("conv"):
        window = c["B"] * (c["W"] - 1) * c["C"] * es if c["state"] else 0
        params = c["C"] * (c["W"] + 1) * 4
        if c["op"] == "conv_grad":
            return {"bytes": 3 * rows * es + 2 * params + 3 * window, "flops": rows * (6 * c["W"] + 12)}
        return {"bytes": 2 * rows * es + params + 2 * window, "flops": rows * (2 * c["W"] + 6)}
    shared = 2 * tokens * c["G"] * c["n"] * es
    params = c["C"] * (c["n"] + 2) * 4
    state = c["B"] * c["C"] * c["n"] * 4 if c["state"] else 0
    wide = 3 if c["gate"] else 2  # x, delta and z
    if c["op"] == "ssm_grad":
        return {"bytes": (2 * wide + 1) * rows * es + 2 * shared + 2 * params + 3 * state,
                "flops": rows * (20 * c["n"] + 30)}
    return {"bytes": (wide + 1) * rows * es + shared + params + 2 * state, "flops": rows * (7 * c["n"] + 16)}


# ---- 64 bits, token by token -----------------------------------------------

def _lengths_of(s):
    c = s["case"]
    return torch.full((c["B"],), c["N"], device="cuda") if s["lengths"] is None else s["lengths"].long()


def _gate_value(u):
    """silu and its slope."""
    sig = 1.0 / (1.0 + torch.exp(-u))
    return u * sig, sig + u * sig * (1.0 - sig)


def _exact_conv(s):
    c = s["case"]
    B, N, C, W = c["B"], c["N"], c["C"], c["W"]
    if c["op"] == "conv_step":
        N = 1
    before = s["S0"].double() if c["state"] else torch.zeros(B, W - 1, C, dtype=torch.float64, device="cuda")
    x = s["x"].double().reshape(B, N, C)
    seen = torch.empty(B, W - 1 + N, C, dtype=torch.float64, device="cuda")
    seen[:, :W - 1], seen[:, W - 1:] = before, x
    w = s["weight"].double()
    u = s["bias"].double().expand(B, N, C).clone()
    for j in range(W):
        u.addcmul_(seen[:, j:j + N], w[:, j])
    value, slope = _gate_value(u) if c["act"] == "silu" else (u, torch.ones_like(u))
    ends = _lengths_of(s).tolist() if c["op"] != "conv_step" else [1] * B
    last = torch.stack([seen[b, e:e + W - 1] for b, e in enumerate(ends)])
    if c["op"] == "conv_step":
        return {"y": value[:, 0], "S": last}
    for b, e in enumerate(ends):
        value[b, e:] = 0
    if c["op"] == "conv":
        y = value.view(B, N, c["heads"], -1).movedim(2, 1) if c["heads"] else value
        return {"y": y, "S": last} if c["state"] else {"y": y}
    dy = s["dy"].double()
    du = (dy.movedim(1, 2).reshape(B, N, C) if c["heads"] else dy) * slope
    for b, e in enumerate(ends):
        du[b, e:] = 0
    dseen = torch.zeros_like(seen)
    dw = torch.empty_like(w)
    for j in range(W):
        dseen[:, j:j + N].addcmul_(du, w[:, j])
        dw[:, j] = (du * seen[:, j:j + N]).sum((0, 1))
    if c["state"]:
        for b, e in enumerate(ends):
            dseen[b, e:e + W - 1] += s["dS"][b].double()
    r = {"dx": dseen[:, W - 1:], "dweight": dw, "dbias": du.sum((0, 1))}
    return dict(r, dS0=dseen[:, :W - 1]) if c["state"] else r


def _exact_ssm(s):
    c = s["case"]
    B, N, C, n, G = c["B"], c["N"], c["C"], c["n"], c["G"]
    step = c["op"] == "ssm_step"

    def tokens(t):
        return t.double()[None] if step else t.double().movedim(1, 0)

    x, raw, Bm, Cm = (tokens(s[m]) for m in ("x", "delta", "Bm", "Cm"))
    group = torch.arange(C, device="cuda") * G // C
    A, D, ends = s["A"].double(), s["D"].double(), _lengths_of(s)
    pre = raw + s["delta_bias"].double()
    dt = torch.logaddexp(pre, torch.zeros_like(pre))
    gate, slope = _gate_value(tokens(s["z"])) if s["z"] is not None else (None, None)
    S = s["S0"].double() if c["state"] else torch.zeros(B, C, n, dtype=torch.float64, device="cuda")

    def token(t, S):
        """(decayed state, state after token t, whether each row has the token)."""
        on = (t < ends)[:, None, None]
        kept = torch.exp(dt[t][..., None] * A) * S
        return kept, torch.where(on, kept + (dt[t] * x[t])[..., None] * Bm[t][:, group], S), on

    if c["op"] != "ssm_grad":
        out = torch.empty_like(x)
        for t in range(N):
            _, S, on = token(t, S)
            y = (S * Cm[t][:, group]).sum(-1) + D * x[t]
            out[t] = torch.where(on[..., 0], y if gate is None else y * gate[t], torch.zeros_like(y))
        if step:
            return {"out": out[0], "S": S}
        return {"out": out.movedim(0, 1), "S": S} if c["state"] else {"out": out.movedim(0, 1)}
    every, starts = 64, []
    for t in range(N):
        if t % every == 0:
            starts.append(S)
        _, S, _ = token(t, S)
    dout = s["dout"].double().movedim(1, 0)
    dS = s["dS"].double() if c["state"] else torch.zeros_like(S)
    dx, ddelta, dz = torch.zeros_like(x), torch.zeros_like(x), torch.zeros_like(x)
    dB, dC = torch.zeros_like(Bm), torch.zeros_like(Cm)
    dA, dD, dbias = torch.zeros_like(A), torch.zeros_like(D), torch.zeros_like(D)

    def over_group(t):
        return t.view(B, G, C // G, n).sum(2)

    for i in reversed(range(len(starts))):
        S, kept = starts[i], []
        for t in range(i * every, min(N, (i + 1) * every)):
            held, S, on = token(t, S)
            kept.append((held, S, on))
        for t in reversed(range(i * every, min(N, (i + 1) * every))):
            held, S, on = kept[t - i * every]
            b_row, c_row, on1 = Bm[t][:, group], Cm[t][:, group], on[..., 0]
            dy = torch.where(on1, dout[t], torch.zeros_like(dout[t]))
            if gate is not None:
                dz[t] = dy * ((S * c_row).sum(-1) + D * x[t]) * slope[t]
                dy = dy * gate[t]
            dC[t] = over_group(dy[..., None] * S)
            dS = dS + dy[..., None] * c_row
            here = torch.where(on, dS, torch.zeros_like(dS))
            through = here * held  # of dt A
            written = (here * b_row).sum(-1)  # of dt x
            ddt = (through * A).sum(-1) + written * x[t]
            dA += (through * dt[t][..., None]).sum(0)
            dx[t] = written * dt[t] + D * dy
            dD += (dy * x[t]).sum(0)
            dB[t] = over_group(here * (dt[t] * x[t])[..., None])
            ddelta[t] = ddt / (1.0 + torch.exp(-pre[t]))
            dbias += ddelta[t].sum(0)
            dS = torch.where(on, dS * torch.exp(dt[t][..., None] * A), dS)
    r = {"dx": dx.movedim(0, 1), "ddelta": ddelta.movedim(0, 1), "dA": dA, "dBm": dB.movedim(0, 1),
         "dCm": dC.movedim(0, 1), "dD": dD}
    if gate is not None:
        r["dz"] = dz.movedim(0, 1)
    r["ddelta_bias"] = dbias
    return dict(r, dS0=dS) if c["state"] else r


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_conv(s) if case["op"].startswith("conv") else _exact_ssm(s)
