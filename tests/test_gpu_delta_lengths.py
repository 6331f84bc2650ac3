"""The gated delta rule with keys of any length (feature_map "none").

The recurrence is stable while beta |k|^2 <= 2, so a short key goes with a large
beta.  Scaling k_t by c and beta_t by 1 / c^2 multiplies the state's rows by no
common factor where c varies, but what is written for a token and read under its
own key keeps its size, so the bounds are those of keys of length one: fp32
results 1e-5 of the 2-norm and of the largest entry (two fp16 parts of an
operand leave 2^-22 = 2.4e-7 per term), bf16 results 2^-8 of a value for their
own rounding and as much again for the terms' 2^-12 and for sums of 128.
"""
import numpy as np
import pytest
import torch

from delta_bounds import excess, within
from gpu_util import to_np
from oracle import delta

pytestmark = pytest.mark.gpu

la = pytest.importorskip("kernelised_causal_linear_gb300")

BF, F32 = torch.bfloat16, torch.float32
INPUTS = ("q", "k", "v", "beta", "log_alpha")
NAMES = ("dq", "dk", "dv", "dbeta", "dlog_alpha", "dS0")


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.fail("GPU test run without a CUDA device")
    yield
    assert la.la_get_device_status() == 0


def problem(N, lengths, writing, seed, dtype=BF, d=64, dv=64, B=1, H=4, Hk=2, gated=True):
    """Keys of unit direction, half of it shared, times lengths [B,Hk,N]; beta = writing / |k|^2."""
    g = torch.Generator().manual_seed(3000 + seed)
    n = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    k = n(B, Hk, N, d) + n(1, Hk, 1, d)
    k = (k / k.norm(dim=-1, keepdim=True) * lengths[..., None]).to(dtype)
    p = dict(q=n(B, Hk, N, d).to(dtype), k=k, v=n(B, H, N, dv).to(dtype),
             beta=(writing / k.float().square().sum(-1)).repeat_interleave(H // Hk, 1),
             log_alpha=-torch.nn.functional.softplus(n(B, H, N) - 2) if gated else None,
             S0=None, dout=n(B, H, N, dv).to(dtype), dS_out=None)
    return {a: None if x is None else x.cuda().contiguous() for a, x in p.items()}


def errors(got, ref):
    """2-norm and largest entry of the error, and the worst token's 2-norm."""
    g, r = to_np(got), np.asarray(ref)
    assert g.shape == r.shape and np.all(np.isfinite(g))
    e = g - r
    rows = np.linalg.norm(e, axis=-1) / np.maximum(np.linalg.norm(r, axis=-1), 1e-30)
    return np.linalg.norm(e) / np.linalg.norm(r), np.abs(e).max() / np.abs(r).max(), rows.max()


def check(p, rows=()):
    """rows: the results whose tokens are also judged one by one, where they are bf16."""
    h = lambda n: None if p[n] is None else to_np(p[n])  # noqa: E731
    scale = p["q"].shape[-1] ** -0.5
    args = [p[n] for n in INPUTS]
    got = dict(zip(("out", "S"), la.la_forward_delta(*args, feature_map="none", return_state=True)))
    ref = dict(zip(("out", "S"), delta.forward(*map(h, INPUTS), scale=scale, l2=False)))
    got.update(zip(NAMES, la.la_backward_delta(p["dout"], *args, feature_map="none")))
    ref.update(zip(NAMES, delta.backward(h("dout"), *map(h, INPUTS), scale=scale, l2=False)))
    for name, g in got.items():
        if g is None or name == "dS0":
            continue
        two, most, row = errors(g, ref[name])
        print(f"{name}: 2-norm {two:.2e}, largest {most:.2e}, worst token {row:.2e}")
        bound = 1e-5 if g.dtype == F32 else 2 * 2.0 ** -8
        assert two <= bound and most <= bound, (name, two, most)
        if name in rows and g.dtype == BF:  # an fp32 row may hang on one dot product that cancels
            assert row <= bound, (name, row)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("N", [16, 17, 64, 65, 200])
@pytest.mark.parametrize("length,writing", [(2.0 ** -6, 1.0), (0.01, 1.0), (0.01, 1.9), (100.0, 1.0)])
def test_short_and_long_keys(N, length, writing, dtype):
    """beta |k|^2 = 1 with beta = 4096 or 1e4 or 1e-4: as stable as unit keys with beta = 1."""
    check(problem(N, torch.full((1, 2, N), length), writing, N, dtype), rows=("out", "dv"))


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("least", [1e-2, 1e-3, 1e-4])
@pytest.mark.parametrize("N,d,dv", [(64, 64, 64), (150, 128, 128), (700, 32, 64)])
def test_keys_of_mixed_lengths(N, d, dv, least, dtype):
    """Lengths spread over 1 .. 1e-4 in one chunk, beta = 1 / |k|^2 (normalised writing)."""
    g = torch.Generator().manual_seed(N)
    lengths = torch.exp(torch.rand(1, 2, N, generator=g) * float(np.log(least)))
    p = problem(N, lengths, 1.0, N + 1, dtype, d, dv)
    check(p, rows=("dv",))


def beyond(p):
    """Outside the stable range results grow by orders of magnitude within a chunk: they are finite while
    fp32 holds them, and of a chunk's largest values as right as bf16 numbers are (2 x 2^-8)."""
    h = lambda n: None if p[n] is None else to_np(p[n])  # noqa: E731
    scale = p["q"].shape[-1] ** -0.5
    args = [p[n] for n in INPUTS]
    got = list(la.la_forward_delta(*args, feature_map="none", return_state=True))
    ref = list(delta.forward(*map(h, INPUTS), scale=scale, l2=False))
    got += la.la_backward_delta(p["dout"], *args, feature_map="none")
    ref += delta.backward(h("dout"), *map(h, INPUTS), scale=scale, l2=False)
    for name, g, r in zip(("out", "S") + NAMES, got, ref):
        if g is not None:
            two, most, _ = errors(g, r)
            print(f"{name}: 2-norm {two:.2e}, largest {most:.2e}")
            assert two <= 2 * 2.0 ** -8 and most <= 2 * 2.0 ** -8, (name, two, most)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("N", [17, 64, 100, 130])
@pytest.mark.parametrize("writing", [2.2, 2.5])
def test_a_repeated_key_that_grows(N, writing, dtype):
    """One key everywhere: the state's row is multiplied by 1 - beta |k|^2 = -1.2 or -1.5 at each token,
    1e5 or 1e11 over a chunk."""
    p = problem(N, torch.ones(1, 2, N), writing, 5, dtype, gated=False)
    p["k"][:] = p["k"][:, :, :1]
    beyond(p)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("at", [3, 30, 63])
def test_one_token_writes_far_too_strongly(at, dtype):
    """beta |k|^2 = 1e4 at one token among ones."""
    p = problem(100, torch.ones(1, 2, 100), 1.0, 6 + at, dtype)
    p["beta"][:, :, at] *= 1e4
    beyond(p)


@pytest.mark.parametrize("N,d,dv", [(64, 128, 128), (129, 32, 32), (200, 64, 64)])
def test_keys_of_six_orders_of_magnitude(N, d, dv):
    """Lengths spread over 1 .. 1e-6: dv is fp32 until its rounding (delta_bounds), dbeta and S stay fp32."""
    g = torch.Generator().manual_seed(N)
    p = problem(N, torch.exp(-14 * torch.rand(1, 2, N, generator=g)), 1.9, N + 2, BF, d, dv, gated=False)
    h = lambda n: None if p[n] is None else to_np(p[n])  # noqa: E731
    args = [p[n] for n in INPUTS]
    got = la.la_backward_delta(p["dout"], *args, feature_map="none")
    ref = delta.backward(h("dout"), *map(h, INPUTS), scale=d ** -0.5, l2=False)
    print(f"dv {excess(to_np(got[2]), ref[2]):.2f} parts, dbeta {errors(got[3], ref[3])[0]:.2e}")
    assert within("dv", to_np(got[2]), ref[2])
    assert errors(got[3], ref[3])[0] <= 1e-5
    S = la.la_forward_delta(*args, feature_map="none", return_state=True)[1]
    assert errors(S, delta.forward(*map(h, INPUTS), scale=d ** -0.5, l2=False)[1])[0] <= 1e-5
