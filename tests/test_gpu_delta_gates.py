"""dlog_alpha token by token, for gates of every strength.

dlog_alpha_t = <S'_t, dS'_t> with S'_t = a_t S_{t-1} the decayed state and dS'_t its
gradient.  Both are held to the library's fp32 bound, 1e-5 of their 2-norm, so
their product is off by at most about 1e-5 |S'_t| |dS'_t| (twice that, less the
independence of the two: both measure near 1e-6).  S'_t carries a_t, so a strong
gate's gradient is small, and right to its own size."""
import numpy as np
import pytest
import torch

from gpu_util import to_np

pytestmark = pytest.mark.gpu

la = pytest.importorskip("kernelised_causal_linear_gb300")

BF, F32 = torch.bfloat16, torch.float32
DTYPES = [F32, BF]
INPUTS = ("q", "k", "v", "beta", "log_alpha")


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.fail("GPU test run without a CUDA device")
    yield
    assert la.la_get_device_status() == 0


def problem(B, H, Hk, N, d, dv, dtype, seed, state=True):
    g = torch.Generator().manual_seed(4000 + seed)
    n = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    p = dict(q=n(B, Hk, N, d).to(dtype), k=n(B, Hk, N, d).to(dtype), v=n(B, H, N, dv).to(dtype),
             beta=torch.sigmoid(n(B, H, N)), log_alpha=torch.zeros(B, H, N),
             S0=0.3 * n(B, H, d, dv) if state else None, dout=n(B, H, N, dv).to(dtype),
             dS_out=0.3 * n(B, H, d, dv) if state else None)
    return {a: None if x is None else x.cuda().contiguous() for a, x in p.items()}


def reference(p):
    """dlog_alpha and |S'_t| |dS'_t| in 64 bits, token by token."""
    H = p["v"].shape[1]
    unit = lambda x: x / np.sqrt((x * x).sum(-1, keepdims=True) + 1e-6)  # noqa: E731
    heads = lambda n: np.repeat(unit(to_np(p[n])), H // p[n].shape[1], axis=1)  # noqa: E731
    q, k = heads("q") * p["q"].shape[-1] ** -0.5, heads("k")
    v, b, a, do = to_np(p["v"]), to_np(p["beta"]), np.exp(to_np(p["log_alpha"])), to_np(p["dout"])
    B, _, N, dv = v.shape
    zero = np.zeros((B, H, k.shape[-1], dv))
    S = zero if p["S0"] is None else to_np(p["S0"])
    kept = []
    for t in range(N):
        Sd = S * a[:, :, t, None, None]
        e = v[:, :, t] - np.einsum("bhij,bhi->bhj", Sd, k[:, :, t])
        S = Sd + np.einsum("bhi,bhj->bhij", k[:, :, t], b[:, :, t, None] * e)
        kept.append(Sd)
    dS = zero if p["dS_out"] is None else to_np(p["dS_out"])
    dg, mag = np.zeros_like(b), np.zeros_like(b)
    for t in reversed(range(N)):
        dS = dS + np.einsum("bhi,bhj->bhij", q[:, :, t], do[:, :, t])
        du = np.einsum("bhij,bhi->bhj", dS, k[:, :, t])
        dS = dS - np.einsum("bhi,bhj->bhij", k[:, :, t], b[:, :, t, None] * du)
        dg[:, :, t] = (dS * kept[t]).sum((-1, -2))
        mag[:, :, t] = np.sqrt((dS ** 2).sum((-1, -2)) * (kept[t] ** 2).sum((-1, -2)))
        dS = dS * a[:, :, t, None, None]
    return dg, mag


def check(p):
    got = la.la_backward_delta(p["dout"], *(p[n] for n in INPUTS), S0=p["S0"], dS_out=p["dS_out"])[4]
    ref, mag = reference(p)
    g = to_np(got)
    assert np.all(np.isfinite(g))
    off = np.abs(g - ref) / np.maximum(mag, 1e-30)
    print(f"worst token {off.max():.2e}")
    assert np.all(np.abs(g - ref) <= 1e-5 * mag + 1e-30), off.max()
    return g


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("N", [1, 2, 33, 64, 65, 130])
@pytest.mark.parametrize("gate", [-1.0, -4.0, -8.0, -12.0, -16.0, -30.0])
def test_every_gate_as_strong(gate, N, dtype):
    p = problem(2, 4, 2, N, 64, 64, dtype, N)
    p["log_alpha"][:] = gate
    check(p)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("at", [0, 1, 31, 32, 63, 64, 99])
def test_one_strong_gate_among_weak_ones(at, dtype):
    p = problem(2, 4, 2, 100, 64, 32, dtype, at)
    p["log_alpha"][:] = -0.01
    p["log_alpha"][:, :, at] = -16.0
    check(p)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("d,dv", [(32, 32), (32, 128), (64, 64), (128, 32), (128, 128)])
@pytest.mark.parametrize("state", [False, True])
def test_gates_of_every_size_mixed(d, dv, state, dtype):
    p = problem(2, 4, 1, 200, d, dv, dtype, d + dv, state)
    g = torch.Generator().manual_seed(d + 2 * dv)
    kinds = torch.tensor([0.0, -1e-3, -0.5, -4.0, -8.0, -16.0, -25.0])
    p["log_alpha"] = kinds[torch.randint(0, 7, (2, 4, 200), generator=g)].cuda()
    p["beta"] = torch.tensor([0.0, 0.3, 1.0, 2.0])[torch.randint(0, 4, (2, 4, 200), generator=g)].cuda()
    check(p)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("gate", [-129.0, -1000.0, -float("inf")])
def test_a_reset_has_no_gradient(gate, dtype):
    """Every second gate a reset, then all of them: exactly 0 there."""
    p = problem(2, 2, 2, 130, 64, 64, dtype, 7)
    p["log_alpha"][:] = -0.1
    p["log_alpha"][:, :, ::2] = gate
    g = check(p)
    assert (g[:, :, ::2] == 0).all() and (g[:, :, 1::2] != 0).any()
    p["log_alpha"][:] = gate
    assert (check(p) == 0).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("gate", [-0.05, -8.0])
def test_strong_gates_in_segments(gate, dtype):
    """One head over many chunks, cut into segments that run at once."""
    p = problem(1, 1, 1, 1100, 64, 64, dtype, 8)
    p["log_alpha"][:] = gate
    p["log_alpha"][:, :, 5::97] = -16.0
    check(p)
