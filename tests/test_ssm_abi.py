"""Argument errors of the convolution and scan entry points: every one comes back before
anything touches a GPU (the pointers below are never followed)."""
import ctypes

import pytest
import torch

FAKE, ODD, BYTE = 0x10000, 0x10004, 0x10001
INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 6


@pytest.fixture(scope="module")
def lib():
    from kernelised_causal_linear_gb300 import build

    build.build()
    from kernelised_causal_linear_gb300 import _binding

    return _binding.raw


def call(fn, order, sizes, given, tail=()):
    args = dict(order)
    for n, x in given.items():
        assert n in args or n in sizes, n
        (args if n in args else sizes)[n] = x
    return fn(*args.values(), *sizes.values(), *tail, None)


def conv(lib, **kw):
    order = dict(x=FAKE, xb=8, xt=8, weight=FAKE, bias=FAKE, y=FAKE, S0=FAKE, S_out=FAKE, lengths=FAKE)
    return call(lib.la_forward_conv, order, dict(B=2, N=8, C=16, H=2, W=4, act=0, dtype=0), kw)


def conv_step(lib, **kw):
    order = dict(S=FAKE, x=FAKE, xb=8, weight=FAKE, bias=FAKE, y=FAKE)
    return call(lib.la_decode_step_conv, order, dict(B=2, C=16, W=4, act=0, dtype=0), kw)


def conv_grad(lib, ws=FAKE, ws_bytes=1 << 40, **kw):
    order = dict(dy=FAKE, dS_out=FAKE, x=FAKE, xb=8, xt=8, weight=FAKE, bias=FAKE, S0=FAKE, lengths=FAKE, dx=FAKE,
                 dweight=FAKE, dbias=FAKE, dS0=FAKE)
    return call(lib.la_backward_conv, order, dict(B=2, N=8, C=16, H=2, W=4, act=0, dtype=0), kw, (ws, ws_bytes))


def strides(*s):
    return (ctypes.c_int64 * len(s))(*s)


SSM = dict(B=2, N=8, C=16, G=2, n=16, softplus=1, dtype=0)


def ssm(lib, ws=FAKE, ws_bytes=1 << 40, **kw):
    order = dict.fromkeys(("x", "delta", "A", "Bm", "Cm", "D", "z", "bias", "out", "S0", "S_out", "lengths"), FAKE)
    order["strides"] = None
    return call(lib.la_forward_ssm, order, dict(SSM), kw, (ws, ws_bytes))


def ssm_step(lib, **kw):
    order = dict.fromkeys(("S", "x", "delta", "A", "Bm", "Cm", "D", "z", "bias", "out"), FAKE)
    order["strides"] = None
    return call(lib.la_decode_step_ssm, order, {k: v for k, v in SSM.items() if k != "N"}, kw)


def ssm_grad(lib, ws=FAKE, ws_bytes=1 << 40, **kw):
    order = dict.fromkeys(("dout", "dS_out", "x", "delta", "A", "Bm", "Cm", "D", "z", "bias", "S0", "lengths", "dx",
                           "ddelta", "dA", "dBm", "dCm", "dD", "dz", "dbias", "dS0"), FAKE)
    order["strides"] = None
    return call(lib.la_backward_ssm, order, dict(SSM), kw, (ws, ws_bytes))


BAD_CONV = [(dict(B=0), INVALID), (dict(C=0), INVALID), (dict(W=0), INVALID), (dict(W=1), UNSUPPORTED),
            (dict(W=5), UNSUPPORTED), (dict(act=3), INVALID), (dict(dtype=2), INVALID), (dict(xb=-1), INVALID),
            (dict(C=1 << 25), UNSUPPORTED), (dict(B=1 << 40), UNSUPPORTED), (dict(x=None), INVALID),
            (dict(x=BYTE), INVALID), (dict(weight=None), INVALID), (dict(weight=ODD), INVALID),
            (dict(bias=ODD), INVALID)]


@pytest.mark.parametrize("kw,code", BAD_CONV, ids=[str(c[0]) for c in BAD_CONV])
def test_every_conv_call_refuses(lib, kw, code):
    assert conv(lib, **kw) == code
    assert conv_step(lib, **kw) == code
    assert conv_grad(lib, **kw) == code


def test_conv_refusals(lib):
    for kw in (dict(N=-1), dict(H=0), dict(H=3), dict(xt=-1), dict(y=None), dict(y=ODD), dict(S0=ODD),
               dict(S_out=ODD), dict(lengths=BYTE)):
        assert conv(lib, **kw) == INVALID, kw
    assert conv(lib, N=1 << 33) == UNSUPPORTED
    for kw in (dict(S=None), dict(S=ODD), dict(y=None), dict(y=ODD)):
        assert conv_step(lib, **kw) == INVALID, kw
    for kw in (dict(N=-1), dict(H=3), dict(dy=None), dict(dy=ODD), dict(dx=None), dict(dweight=None),
               dict(dbias=None), dict(bias=None), dict(dS0=ODD), dict(dS_out=ODD), dict(S0=ODD), dict(lengths=BYTE)):
        assert conv_grad(lib, **kw) == INVALID, kw
    need = lib.la_conv_backward_workspace_size(2, 8, 16, 4, 0)
    assert need > 0
    assert conv_grad(lib, ws=None) == WORKSPACE
    assert conv_grad(lib, ws_bytes=need - 1) == WORKSPACE
    assert conv_grad(lib, ws=FAKE + 128) == WORKSPACE


BAD_SSM = [(dict(B=0), INVALID), (dict(C=0), INVALID), (dict(G=0), INVALID), (dict(G=3), INVALID),
           (dict(n=0), INVALID), (dict(n=4), UNSUPPORTED), (dict(n=128), UNSUPPORTED), (dict(softplus=2), INVALID),
           (dict(dtype=-1), INVALID), (dict(C=1 << 25), UNSUPPORTED), (dict(B=1 << 40), UNSUPPORTED),
           (dict(x=None), INVALID), (dict(x=BYTE), INVALID), (dict(delta=None), INVALID), (dict(A=None), INVALID),
           (dict(A=ODD), INVALID), (dict(Bm=None), INVALID), (dict(Cm=BYTE), INVALID), (dict(D=ODD), INVALID),
           (dict(z=BYTE), INVALID), (dict(bias=ODD), INVALID)]


@pytest.mark.parametrize("kw,code", BAD_SSM, ids=[str(c[0]) for c in BAD_SSM])
def test_every_ssm_call_refuses(lib, kw, code):
    assert ssm(lib, **kw) == code
    assert ssm_step(lib, **kw) == code
    assert ssm_grad(lib, **kw) == code


def test_ssm_refusals(lib):
    for kw in (dict(N=-1), dict(out=None), dict(out=ODD), dict(S0=ODD), dict(S_out=ODD), dict(lengths=BYTE),
               dict(strides=strides(*[8] * 9, -1))):
        assert ssm(lib, **kw) == INVALID, kw
    assert ssm(lib, N=1 << 33) == UNSUPPORTED
    long = lib.la_ssm_workspace_size(2, 100000, 16, 2, 16, 0)
    assert long > 0
    assert ssm(lib, N=100000, ws=None) == WORKSPACE
    assert ssm(lib, N=100000, ws_bytes=long - 1) == WORKSPACE
    assert ssm(lib, N=100000, ws=FAKE + 16) == WORKSPACE
    for kw in (dict(S=None), dict(S=ODD), dict(out=None), dict(out=ODD), dict(strides=strides(8, 8, -1, 8, 8))):
        assert ssm_step(lib, **kw) == INVALID, kw
    for kw in (dict(N=-1), dict(dout=None), dict(dout=BYTE), dict(dS_out=ODD), dict(dx=None), dict(ddelta=None),
               dict(dA=None), dict(dBm=None), dict(dCm=ODD), dict(dD=None), dict(D=None), dict(dz=None),
               dict(z=None), dict(dbias=None), dict(bias=None), dict(dS0=ODD), dict(S0=ODD),
               dict(strides=strides(*[8] * 11, -1))):
        assert ssm_grad(lib, **kw) == INVALID, kw
    need = lib.la_ssm_backward_workspace_size(2, 8, 16, 2, 16, 0)
    assert need > 0
    assert ssm_grad(lib, ws=None) == WORKSPACE
    assert ssm_grad(lib, ws_bytes=need - 1) == WORKSPACE


def test_workspace_sizes(lib):
    assert lib.la_ssm_workspace_size(2, 0, 16, 1, 16, 0) == 0
    assert lib.la_ssm_backward_workspace_size(2, 0, 16, 1, 16, 0) == 0
    assert lib.la_ssm_backward_workspace_size(2, 8, 16, 3, 16, 0) == 0
    assert lib.la_conv_backward_workspace_size(2, 0, 16, 4, 0) == 0
    assert lib.la_conv_backward_workspace_size(2, 8, 16, 7, 0) == 0


def test_binding_refuses_cpu_tensors():
    import kernelised_causal_linear_gb300 as la

    x, w = torch.zeros(1, 4, 16), torch.zeros(16, 4)
    A, bc = torch.zeros(16, 16), torch.zeros(1, 4, 1, 16)
    for f in (lambda: la.la_forward_conv(x, w), lambda: la.la_backward_conv(x, x, w),
              lambda: la.la_decode_step_conv(torch.zeros(1, 3, 16), x[:, 0], w),
              lambda: la.la_forward_ssm(x, x, A, bc, bc), lambda: la.la_backward_ssm(x, x, x, A, bc, bc),
              lambda: la.la_decode_step_ssm(torch.zeros(1, 16, 16), x[:, 0], x[:, 0], A, bc[:, 0], bc[:, 0])):
        with pytest.raises(ValueError):
            f()
