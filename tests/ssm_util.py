"""Inputs, calls and comparisons of the convolution and scan tests (imported only by tests).

Tolerances.
 - fp32 results: 1e-5 of the tensor's 2-norm and of its largest entry, the library's bound.
   A decay is off by at most 2.4 * 2^-24 and by 0.29 * 2^-24 in the mean; a state adds up
   at most N of the mean ones: N 1.7e-8, under 7e-6 for N up to 400 (longer tests say what
   they take).  A step is off by a few 2^-24 and everything else is fp32 sums.
 - a bf16 result is rounded once besides, 2^-8 of its value at most."""
import numpy as np
import torch

import kernelised_causal_linear_gb300 as la
from gpu_util import to_np
from oracle import ssm

BF, F32 = torch.bfloat16, torch.float32
LEAVES = ("x", "delta", "A", "Bm", "Cm", "D", "z", "delta_bias", "S0")


def near(got, ref, what, tol=1e-5):
    g, r = to_np(got), np.asarray(ref)
    assert g.shape == r.shape, (what, g.shape, r.shape)
    assert np.all(np.isfinite(g)), what
    if not g.size:
        return
    e, most = np.abs(g - r), np.abs(r).max()
    half = 2.0 ** -8 if got.dtype == BF else 0.0
    assert np.all(e <= half * np.abs(r) + tol * most), (what, e.max(), most)
    if not half:
        assert np.linalg.norm(e) <= tol * np.linalg.norm(r), (what, np.linalg.norm(e) / np.linalg.norm(r))


def np_or_none(t):
    return None if t is None else to_np(t)


def ssm_problem(B, N, C, n=16, G=1, dtype=F32, seed=0, gate=True, state=True, extras=True, lengths=None,
                slices=False, low=1e-3):
    g = torch.Generator().manual_seed(3000 + seed)
    m = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    step = torch.exp(torch.rand(C, generator=g) * (np.log(0.1) - np.log(low)) + np.log(low))
    p = dict(x=m(B, N, C).to(dtype), delta=(0.5 * m(B, N, C)).to(dtype),
             A=-torch.exp(torch.log(torch.arange(1, n + 1.0)) + 0.2 * m(C, n)), Bm=m(B, N, G, n).to(dtype),
             Cm=m(B, N, G, n).to(dtype), D=m(C) if extras else None, z=m(B, N, C).to(dtype) if gate else None,
             delta_bias=step + torch.log(-torch.expm1(-step)) if extras else None,
             S0=0.3 * m(B, C, n) if state else None, dout=m(B, N, C).to(dtype),
             dS_out=0.3 * m(B, C, n) if state else None)
    if not extras:
        p["delta"] = p["delta"] - 4
    p = {k: None if v is None else v.cuda() for k, v in p.items()}
    if slices:  # wide rows, the inputs somewhere inside
        for k in ("x", "z", "delta", "dout"):
            if p[k] is not None:
                p[k] = torch.cat([p[k][..., :slices], p[k], p[k]], -1)[..., slices:slices + C]
        both = torch.cat([p["x"][..., :slices], p["Bm"].flatten(2), p["Cm"].flatten(2)], -1)
        p["Bm"] = both[..., slices:slices + G * n].unflatten(-1, (G, n))
        p["Cm"] = both[..., slices + G * n:].unflatten(-1, (G, n))
    p["lengths"] = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")
    return p


def ssm_args(p):
    return [p[k] for k in ("x", "delta", "A", "Bm", "Cm")], {k: p[k] for k in ("D", "z", "delta_bias")}


def ssm_oracle(p, softplus=True, grad=False):
    pos, kw = ssm_args(p)
    more = dict(dout=to_np(p["dout"]), dS_out=np_or_none(p["dS_out"])) if grad else {}
    return ssm.scan(*map(to_np, pos), **{k: np_or_none(v) for k, v in kw.items()}, softplus_on=softplus,
                    S0=np_or_none(p["S0"]), lengths=np_or_none(p["lengths"]), **more)


def check_ssm(p, softplus=True, grad=True, tol=1e-5):
    pos, kw = ssm_args(p)
    out, S = la.la_forward_ssm(*pos, **kw, softplus=softplus, S0=p["S0"], return_state=True, lengths=p["lengths"])
    assert out.dtype == p["x"].dtype and S.dtype == F32
    if not grad:
        r_out, r_S = ssm_oracle(p, softplus)
        near(out, r_out, "out", tol)
        near(S, r_S, "S", tol)
        return
    ref = ssm_oracle(p, softplus, True)
    near(out, ref["out"], "out", tol)
    near(S, ref["S"], "S", tol)
    grads = la.la_backward_ssm(p["dout"], *pos, **kw, softplus=softplus, S0=p["S0"], dS_out=p["dS_out"],
                               lengths=p["lengths"])
    for name, got in zip(LEAVES, grads):
        if p[name] is None:
            assert got is None, name
        else:
            assert got.dtype == p[name].dtype
            near(got, ref[name], "d" + name, tol)


def conv_problem(B, N, C, W=4, dtype=F32, seed=0, heads=None, state=True, bias=True, lengths=None, slices=0):
    g = torch.Generator().manual_seed(4000 + seed)
    m = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    p = dict(x=m(B, N, C).to(dtype), weight=m(C, W), bias=m(C) if bias else None,
             S0=m(B, W - 1, C).to(dtype) if state else None,
             dy=m(*((B, heads, N, C // heads) if heads else (B, N, C))).to(dtype),
             dS_out=m(B, W - 1, C).to(dtype) if state else None)
    p = {k: None if v is None else v.cuda() for k, v in p.items()}
    if slices:
        p["x"] = torch.cat([p["x"][..., :slices], p["x"], p["x"]], -1)[..., slices:slices + C]
    p["lengths"] = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")
    p["heads"] = heads
    return p


def check_conv(p, activation="silu", tol=1e-5):
    heads = p["heads"]
    y, S = la.la_forward_conv(p["x"], p["weight"], p["bias"], activation=activation, heads=heads, S0=p["S0"],
                              return_state=True, lengths=p["lengths"])
    grads = la.la_backward_conv(p["dy"], p["x"], p["weight"], p["bias"], activation=activation, S0=p["S0"],
                                dS_out=p["dS_out"], lengths=p["lengths"])
    dy = to_np(p["dy"])
    if heads:
        dy = np.moveaxis(dy, 1, 2).reshape(p["x"].shape)
    h = {k: np_or_none(p[k]) for k in ("x", "weight", "bias", "S0", "lengths", "dS_out")}
    ry, rS, rdx, rdw, rdb, rdS0 = ssm.conv(h["x"], h["weight"], h["bias"], activation=activation, S0=h["S0"],
                                           lengths=h["lengths"], dy=dy, dS_out=h["dS_out"])
    if heads:
        B, N, C = p["x"].shape
        ry = np.moveaxis(ry.reshape(B, N, heads, C // heads), 2, 1)
    near(y, ry, "y", tol)
    assert np.array_equal(to_np(S), rS)
    for name, got, ref in zip(("dx", "dweight", "dbias", "dS0"), grads, (rdx, rdw, rdb, rdS0)):
        if got is None:
            assert p["bias" if name == "dbias" else "S0"] is None
        else:
            near(got, ref, name, tol)


def same_nan(results, tol=1e-5):
    """(name, got, reference) each: NaN in the same places, and near elsewhere."""
    for name, got, ref in results:
        bad = np.isnan(ref)
        assert np.array_equal(np.isnan(to_np(got)), bad), (name, np.argwhere(np.isnan(to_np(got)) != bad)[:8])
        ok = torch.from_numpy(~bad).to(got.device)
        near(got[ok], np.asarray(ref)[~bad], name, tol)
