"""The short causal convolution where its sizes and rows end, on the GPU against fp64."""
import numpy as np
import pytest
import torch

from gpu_util import to_np
from oracle import ssm

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
@pytest.mark.parametrize("W", [2, 4])
@pytest.mark.parametrize("C", [1, 2, 3, 5])
def test_few_channels(C, W, dtype):
    """Hundreds of block rows for a channel or two: parts in a workspace of exactly the stated size,
    with nothing written behind it.  A sum's longest chain is 25 tokens, 19 parts and 32 joins, each
    term a few 2^-24 off (20 taken): 96 roundings of at most the sum of the terms' sizes, which is at most
    1.1 |dy| |x| (1.1: the largest slope of silu)."""
    u = util()
    p = u.conv_problem(3, 5003, C, W, dtype, 20 + C, lengths=[5003, 4001, 17])
    need = la.la_conv_backward_workspace_size(3, 5003, C, W, dtype)
    ws = torch.randint(0, 256, (need + 65536,), dtype=torch.uint8, device="cuda")
    tail = ws[need:].clone()
    run = lambda **k: la.la_backward_conv(p["dy"], p["x"], p["weight"], p["bias"], S0=p["S0"],  # noqa: E731
                                          dS_out=p["dS_out"], lengths=p["lengths"], **k)
    got = run(workspace=ws[:need])
    assert torch.equal(ws[need:], tail)
    assert all(torch.equal(a, b) for a, b in zip(got, run()))
    h = {k: to_np(p[k]) for k in ("x", "weight", "bias", "S0", "lengths", "dS_out", "dy")}
    _, _, dx, dw, db, dS0 = ssm.conv(h.pop("x"), h.pop("weight"), h.pop("bias"), **h)
    u.near(got[0], dx, "dx")
    u.near(got[3], dS0, "dS0")
    size = lambda *ts: np.sqrt(sum((t.astype(np.float64) ** 2).sum((0, 1)) for t in ts))  # noqa: E731
    terms = 96 * 2.0 ** -24 * 1.1 * size(h["dy"])
    inputs = np.maximum(size(to_np(p["x"]), h["S0"]), np.sqrt(3 * 5003))
    for name, g, want in (("dw", got[1], dw.T), ("db", got[2], db)):
        g = to_np(g).T
        assert np.all(np.abs(g - want) <= terms * inputs), (name, np.abs(g - want).max())


@pytest.mark.parametrize("activation", ["none", "sigmoid"])
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("dtype", [F32, BF])
def test_infinite_last_token_and_the_filters(dtype, W, activation):
    """Where a row's last token is infinite, only the last tap meets it: the others' gradients, the
    bias's and dx stay what they are, for rows that end inside a run and just behind one."""
    u = util()
    lengths = [1, 2, 3, 5, 8, 9, 33, 64, 69, 70]
    p = u.conv_problem(10, 70, 24, W, dtype, 14, lengths=lengths)
    for b, n in enumerate(lengths):
        p["x"][b, n - 1, 0] = float("inf")
    dx, dw, db, dS0 = la.la_backward_conv(p["dy"], p["x"], p["weight"], p["bias"], activation=activation, S0=p["S0"],
                                          dS_out=p["dS_out"], lengths=p["lengths"])
    h = {k: to_np(p[k]) for k in ("x", "weight", "bias", "S0", "lengths", "dS_out", "dy")}
    with np.errstate(invalid="ignore"):
        _, _, rdx, rdw, rdb, rdS0 = ssm.conv(h.pop("x"), h.pop("weight"), h.pop("bias"), activation=activation, **h)
    for got, want, name in ((dx, rdx, "dx"), (dw[:, :-1], rdw[:, :-1], "dw"), (dw[1:], rdw[1:], "dw"), (db, rdb, "db"),
                            (dS0, rdS0, "dS0")):
        u.near(got, want, name)


@pytest.mark.parametrize("activation", ["silu", "sigmoid", "none"])
@pytest.mark.parametrize("dtype", [F32, BF])
def test_nan_of_a_token_is_seen(dtype, activation):
    """A NaN that a row has comes out wherever the definition takes it, and nowhere else."""
    u = util()
    p = u.conv_problem(3, 40, 10, 4, dtype, 15, lengths=[40, 17, 30])
    p["x"][0, 20, 3] = p["x"][1, 16, 4] = p["x"][2, 30, 5] = float("nan")  # the last one behind its row
    y, _ = la.la_forward_conv(p["x"], p["weight"], p["bias"], activation=activation, S0=p["S0"], lengths=p["lengths"])
    got = (y, *la.la_backward_conv(p["dy"], p["x"], p["weight"], p["bias"], activation=activation, S0=p["S0"],
                                   dS_out=p["dS_out"], lengths=p["lengths"]))
    h = {k: to_np(p[k]) for k in ("x", "weight", "bias", "S0", "lengths", "dS_out", "dy")}
    ref = ssm.conv(h.pop("x"), h.pop("weight"), h.pop("bias"), activation=activation, **h)
    u.same_nan(zip(("y", "dx", "dw", "db", "dS0"), got, (ref[0], *ref[2:])))
    win = p["S0"].clone()
    y1 = la.la_decode_step_conv(win, p["x"][:, 20], p["weight"], p["bias"], activation=activation)
    assert torch.isnan(y1).nonzero().tolist() == [[0, 3]]
