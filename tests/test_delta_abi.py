"""Argument errors of the delta-rule and norm entry points: every one comes
back before anything touches a GPU (the pointers below are never followed)."""
import ctypes

import pytest
import torch

I64, I, SZ, VP, F = ctypes.c_int64, ctypes.c_int, ctypes.c_size_t, ctypes.c_void_p, ctypes.c_float
FAKE, ODD = 0x10000, 0x10004
INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 6


@pytest.fixture(scope="module")
def lib():
    from kernelised_causal_linear_gb300 import build

    build.build()
    from kernelised_causal_linear_gb300 import _binding

    return _binding.raw


SIZES = dict(B=1, H=4, Hk=2, N=8, d=64, dv=64, fm=3, scale=1.0, dtype=0)


def forward(lib, ws=FAKE, ws_bytes=1 << 40, **kw):
    p = dict(q=FAKE, k=FAKE, v=FAKE, beta=FAKE, log_alpha=FAKE, out=FAKE, S0=None, S_out=FAKE)
    s = dict(SIZES)
    for n, x in kw.items():
        (p if n in p else s)[n] = x
    return lib.la_forward_delta(*p.values(), *s.values(), ws, ws_bytes, None)


def backward(lib, ws=FAKE, ws_bytes=1 << 40, **kw):
    p = dict.fromkeys(("dout", "dS_out", "q", "k", "v", "beta", "log_alpha", "S0", "dq", "dk",
                       "dv_out", "dbeta", "dlog_alpha", "dS0"), FAKE)
    s = dict(SIZES)
    for n, x in kw.items():
        (p if n in p else s)[n] = x
    return lib.la_backward_delta(*p.values(), *s.values(), ws, ws_bytes, None)


def decode(lib, **kw):
    p = dict.fromkeys(("S", "q", "k", "v", "beta", "log_alpha", "out"), FAKE)
    s = {n: x for n, x in SIZES.items() if n != "N"}
    for n, x in kw.items():
        (p if n in p else s)[n] = x
    return lib.la_decode_step_delta(*p.values(), *s.values(), None)


BAD_SIZES = [(dict(B=0), INVALID), (dict(H=0), INVALID), (dict(Hk=0), INVALID),
             (dict(Hk=3), INVALID), (dict(d=-1), INVALID), (dict(d=48), UNSUPPORTED),
             (dict(dv=256), UNSUPPORTED), (dict(fm=0), UNSUPPORTED), (dict(fm=1), UNSUPPORTED),
             (dict(fm=4), INVALID), (dict(dtype=2), INVALID),
             (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID),
             (dict(B=1 << 40), UNSUPPORTED), (dict(beta=None), INVALID), (dict(beta=ODD), INVALID),
             (dict(q=ODD), INVALID), (dict(k=None), INVALID), (dict(v=ODD), INVALID),
             (dict(log_alpha=ODD), INVALID)]


@pytest.mark.parametrize("kw,code", BAD_SIZES, ids=[str(c[0]) for c in BAD_SIZES])
def test_every_call_refuses(lib, kw, code):
    assert forward(lib, **kw) == code
    assert decode(lib, **kw) == code
    assert backward(lib, **kw) == code


def test_forward_refusals(lib):
    assert forward(lib, N=-1) == INVALID
    assert forward(lib, out=None) == INVALID          # q without out
    assert forward(lib, q=None) == INVALID            # out without q
    assert forward(lib, q=None, out=None, S_out=None) == INVALID
    assert forward(lib, S0=ODD) == INVALID
    assert forward(lib, S_out=ODD) == INVALID
    assert forward(lib, N=1 << 40) == UNSUPPORTED
    need = lib.la_delta_workspace_size(1, 4, 2, 8, 64, 64, 0)
    if need:
        assert forward(lib, ws=None) == WORKSPACE
        assert forward(lib, ws_bytes=need - 1) == WORKSPACE
        assert forward(lib, ws=FAKE + 16) == WORKSPACE


def test_backward_refusals(lib):
    for name in ("dout", "dq", "dk", "dv_out", "dbeta"):
        assert backward(lib, **{name: None}) == INVALID, name
        assert backward(lib, **{name: ODD}) == INVALID, name
    assert backward(lib, log_alpha=None) == INVALID   # dlog_alpha without log_alpha
    assert backward(lib, dlog_alpha=None) == INVALID
    assert backward(lib, dS0=ODD) == INVALID
    assert backward(lib, ws=None) == WORKSPACE
    need = lib.la_delta_backward_workspace_size(1, 4, 2, 8, 64, 64, 0)
    assert need > 0
    assert backward(lib, ws_bytes=need - 1) == WORKSPACE
    assert backward(lib, ws=FAKE + 128) == WORKSPACE


def test_decode_refusals(lib):
    assert decode(lib, S=None) == INVALID
    assert decode(lib, S=ODD) == INVALID
    assert decode(lib, out=None) == INVALID


def norm(lib, grad=False, ws=FAKE, ws_bytes=1 << 40, **kw):
    names = ("dy", "x", "gate", "weight", "dx", "dgate", "dweight") if grad else \
        ("x", "gate", "weight", "y")
    p = dict.fromkeys(names, FAKE)
    s = dict(B=1, H=2, N=4, dv=64, act=0, heads=0, eps=1e-6, x_dtype=0, dtype=0)
    for n, x in kw.items():
        (p if n in p else s)[n] = x
    if grad:
        return lib.la_norm_gate_backward(*p.values(), *s.values(), ws, ws_bytes, None)
    return lib.la_norm_gate(*p.values(), *s.values(), None)


BAD_NORM = [(dict(B=0), INVALID), (dict(N=-1), INVALID), (dict(dv=96), UNSUPPORTED),
            (dict(act=3), INVALID), (dict(heads=2), INVALID), (dict(eps=0.0), INVALID),
            (dict(eps=float("nan")), INVALID), (dict(x_dtype=5), INVALID),
            (dict(dtype=-1), INVALID), (dict(x=None), INVALID), (dict(gate=ODD), INVALID),
            (dict(weight=ODD), INVALID), (dict(N=1 << 40), UNSUPPORTED)]


@pytest.mark.parametrize("kw,code", BAD_NORM, ids=[str(c[0]) for c in BAD_NORM])
def test_norm_refuses(lib, kw, code):
    assert norm(lib, **kw) == code
    assert norm(lib, True, **kw) == code


def test_norm_backward_refusals(lib):
    assert norm(lib, True, dgate=None) == INVALID
    assert norm(lib, True, gate=None) == INVALID
    assert norm(lib, True, dweight=None) == INVALID
    assert norm(lib, True, weight=None) == INVALID
    assert norm(lib, True, dy=None) == INVALID
    assert norm(lib, True, dx=ODD) == INVALID
    assert norm(lib, True, ws=None) == WORKSPACE
    assert norm(lib, True, ws_bytes=16) == WORKSPACE


def test_workspace_sizes(lib):
    f, b = lib.la_delta_workspace_size, lib.la_delta_backward_workspace_size
    assert f(1, 4, 2, 0, 64, 64, 0) == 0 and b(1, 4, 2, 0, 64, 64, 0) == 0
    assert f(1, 4, 3, 8, 64, 64, 0) == 0 and b(1, 4, 3, 8, 64, 64, 0) == 0
    assert 0 < b(1, 4, 2, 100, 64, 64, 0) < b(1, 4, 2, 1000, 64, 64, 0)
    assert lib.la_norm_gate_backward_workspace_size(1, 2, 0, 64) == 0
    assert lib.la_norm_gate_backward_workspace_size(1, 2, 4, 64) > 0


def test_the_other_forwards_do_not_take_l2(lib):
    """LA_FM_L2 belongs to the delta-rule calls."""
    assert lib.la_forward(FAKE, FAKE, FAKE, FAKE, 1, 1, 8, 64, 64, 1, 3, None, 0, FAKE, 1 << 30,
                          None) == INVALID


def test_binding_refuses_cpu_tensors():
    import kernelised_causal_linear_gb300 as la

    q = torch.zeros(1, 1, 4, 64)
    b = torch.zeros(1, 1, 4)
    with pytest.raises(ValueError):
        la.la_forward_delta(q, q, q, b)
    with pytest.raises(ValueError):
        la.la_backward_delta(q, q, q, q, b)
    with pytest.raises(ValueError):
        la.la_decode_step_delta(torch.zeros(1, 1, 64, 64), q[:, :, 0], q[:, :, 0], q[:, :, 0], b[:, :, 0])
    with pytest.raises(ValueError):
        la.la_norm_gate(q)
    with pytest.raises(ValueError):
        la.la_norm_gate_backward(q, q)
