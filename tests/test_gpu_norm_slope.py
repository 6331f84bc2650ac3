"""The gate's slope far from zero, element by element.

sigmoid' = e / (1 + e)^2 with e = exp(-|g|).  Elementwise bound of fp32 results: the
hardware exponential is off by at most 2 + 1.16 |g| ulp (CUDA's stated bound), quotient,
inverse root and the products behind them by a few ulp each, 16 together: in all
(18 + 1.16 |g|) 2^-23 of the value."""
import numpy as np
import pytest
import torch

from gpu_util import to_np
from oracle import delta

pytestmark = pytest.mark.gpu

la = pytest.importorskip("kernelised_causal_linear_gb300")


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.fail("GPU test run without a CUDA device")
    yield
    assert la.la_get_device_status() == 0


@pytest.mark.parametrize("activation", ["silu", "sigmoid"])
@pytest.mark.parametrize("far", [8.0, 12.0, 17.5, 20.0, 40.0])
def test_gradient_of_far_gates(far, activation):
    g = torch.Generator().manual_seed(31)
    n = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    x, dy, w = n(2, 3, 40, 64), n(2, 40, 3, 64), 1 + 0.2 * n(64)
    gate = far + 0.1 * n(2, 40, 3, 64)
    gate[:, ::2] *= -1
    x, gate, w, dy = (t.cuda() for t in (x, gate, w, dy))
    y = la.la_norm_gate(x, gate, w, activation=activation)
    dgate = la.la_norm_gate_backward(dy, x, gate, w, activation=activation)[1]
    # in 64 bits with the slope as e / (1 + e)^2, which does not cancel
    G = to_np(gate)
    e = np.exp(-np.abs(G))
    s, slope = np.where(G >= 0, 1, e) / (1 + e), e / (1 + e) ** 2
    plain = delta.norm_gate(to_np(x), None, to_np(w))  # w xh
    want_y = plain * (G * s if activation == "silu" else s)
    want = to_np(dy) * plain * (s + G * slope if activation == "silu" else slope)
    tol = (18 + 1.16 * np.abs(G)) * 2.0 ** -23
    for got, ref in ((y, want_y), (dgate, want)):
        off = np.abs(to_np(got) - ref) / np.maximum(np.abs(ref), 1e-300)
        print(f"worst element {off.max():.2e}")
        assert np.all(off <= tol), off.max()
