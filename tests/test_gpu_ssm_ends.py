"""The selective scan where rows end, and where what they hold is not finite, on the GPU against
fp64 (tolerances: ssm_util)."""
import pytest
import torch

pytestmark = pytest.mark.gpu

la = pytest.importorskip("kernelised_causal_linear_gb300")
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.fail("GPU test run without a CUDA device")
    yield
    assert la.la_get_device_status() == 0


def util():
    import ssm_util

    return ssm_util


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("n", [8, 16, 32, 64])
@pytest.mark.parametrize("ragged", [True, False])
def test_overflow_of_a_last_state_and_dA(ragged, n, dtype):
    """dA is made of the states before each token: one that the row's last token takes past the
    largest float, from finite inputs, is not among them."""
    u = util()
    for N in (70,) if ragged else (1, 2, 3, 4, 33, 67):
        lengths = [1, 2, 3, 4, 5, 30, 33, 67, 70] if ragged else None
        B = len(lengths) if ragged else 2
        p = u.ssm_problem(B, N, 20, n, 1, dtype, 17 + N, lengths=lengths)
        for b, m in enumerate(lengths or [N] * B):
            p["x"][b, m - 1], p["Bm"][b, m - 1] = 3e38, 1e4
        pos, kw = u.ssm_args(p)
        _, S = la.la_forward_ssm(*pos, **kw, S0=p["S0"], return_state=True, lengths=p["lengths"])
        assert torch.isinf(S).all()
        g = la.la_backward_ssm(p["dout"], *pos, **kw, S0=p["S0"], dS_out=p["dS_out"], lengths=p["lengths"])
        u.near(g[2], u.ssm_oracle(p, grad=True)["A"], "dA")


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("n", [8, 16, 32, 64])
@pytest.mark.parametrize("name", ["z", "x", "delta", "dout", "Bm", "Cm"])
def test_nan_of_a_token_is_seen(name, n, dtype):
    """A NaN that a row has comes out wherever the definition takes it, and nowhere else."""
    u = util()
    p = u.ssm_problem(3, 75, 11, n, 1, dtype, 18, lengths=[75, 40, 61])
    p[name].view(3, 75, -1)[0, 37, 3] = p[name].view(3, 75, -1)[1, 39, 4] = float("nan")
    ref = u.ssm_oracle(p, grad=True)
    p[name].view(3, 75, -1)[2, 61, 5] = float("nan")  # behind its row: not read
    pos, kw = u.ssm_args(p)
    out, S = la.la_forward_ssm(*pos, **kw, S0=p["S0"], return_state=True, lengths=p["lengths"])
    g = la.la_backward_ssm(p["dout"], *pos, **kw, S0=p["S0"], dS_out=p["dS_out"], lengths=p["lengths"])
    u.same_nan([("out", out, ref["out"]), ("S", S, ref["S"])] + [(k, t, ref[k]) for k, t in zip(u.LEAVES, g)])
