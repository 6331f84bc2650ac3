"""bf16 results of the delta rule within their own rounding and what fp16 operands of
one part add (delta_bounds)."""
import pytest
import torch

from delta_bounds import PARTS, excess, within
from gpu_util import to_np
from oracle import delta

pytestmark = pytest.mark.gpu

la = pytest.importorskip("kernelised_causal_linear_gb300")

BF = torch.bfloat16
INPUTS = ("q", "k", "v", "beta", "log_alpha")


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.fail("GPU test run without a CUDA device")
    yield
    assert la.la_get_device_status() == 0


def check(B, H, Hk, N, d, dv, seed, gated=True, state=True, l2=True):
    g = torch.Generator().manual_seed(5000 + seed)
    n = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    qk = 1.0 if l2 else d ** -0.5
    p = dict(q=(n(B, Hk, N, d) * qk).to(BF), k=(n(B, Hk, N, d) * qk).to(BF), v=n(B, H, N, dv).to(BF),
             beta=torch.sigmoid(n(B, H, N)),
             log_alpha=-torch.nn.functional.softplus(2 * n(B, H, N) - 2) if gated else None)
    S0, dS = (0.3 * n(B, H, d, dv), 0.3 * n(B, H, d, dv)) if state else (None, None)
    dout = n(B, H, N, dv).to(BF)
    cuda = lambda t: None if t is None else t.cuda()  # noqa: E731
    host = lambda t: None if t is None else to_np(t)  # noqa: E731
    args, scale, fm = [cuda(p[x]) for x in INPUTS], d ** -0.5, "l2" if l2 else "none"
    got = [la.la_forward_delta(*args, S0=cuda(S0), feature_map=fm)[0],
           *la.la_backward_delta(cuda(dout), *args, S0=cuda(S0), dS_out=cuda(dS), feature_map=fm)[:3]]
    hosts = [host(p[x]) for x in INPUTS]
    ref = [delta.forward(*hosts, scale=scale, l2=l2, S0=host(S0))[0],
           *delta.backward(host(dout), *hosts, scale=scale, l2=l2, S0=host(S0), dS_out=host(dS))[:3]]
    for name, x, y in zip(("out", "dq", "dk", "dv"), map(to_np, got), ref):
        print(f"{name}: {excess(x, y):.2f} of {PARTS[name]} parts")
        assert within(name, x, y), (name, excess(x, y))


@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("dv", [32, 64, 128])
def test_dims(d, dv):
    check(2, 4, 2, 150, d, dv, d + dv)


@pytest.mark.parametrize("gated,state,l2", [(False, False, True), (True, False, False),
                                            (False, True, False), (True, True, True)])
def test_options(gated, state, l2):
    check(2, 6, 1, 200, 128, 64, 7, gated, state, l2)


@pytest.mark.parametrize("B,H,Hk,N,d,dv", [(1, 2, 1, 2500, 128, 128), (10, 16, 8, 100, 64, 128),
                                           (13, 12, 6, 190, 128, 128), (20, 8, 4, 70, 64, 32)])
def test_segments_and_many_heads(B, H, Hk, N, d, dv):
    check(B, H, Hk, N, d, dv, N)
