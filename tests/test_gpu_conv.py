"""The short causal convolution on the GPU against fp64 (tolerances: ssm_util)."""
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
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("B,N,C", [(1, 1, 1), (2, 2, 8), (1, 3, 33), (3, 5, 40), (2, 67, 24), (1, 130, 257),
                                   (700, 5, 8), (2, 70, 66), (1, 9, 2)])
def test_sizes(B, N, C, W, dtype):
    u = util()
    u.check_conv(u.conv_problem(B, N, C, W, dtype, N + C))


@pytest.mark.parametrize("activation", ["silu", "sigmoid", "none"])
@pytest.mark.parametrize("bias", [True, False])
@pytest.mark.parametrize("state", [True, False])
def test_options(activation, bias, state):
    u = util()
    u.check_conv(u.conv_problem(2, 37, 48, 4, F32, 1, bias=bias, state=state), activation)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("heads,C", [(1, 16), (3, 96), (4, 20), (7, 7), (2, 128), (5, 30), (3, 6)])
def test_head_major(heads, C, dtype):
    u = util()
    u.check_conv(u.conv_problem(2, 70, C, 4, dtype, C, heads=heads))


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("W", [2, 4])
def test_lengths(W, dtype):
    """Rows of no, one, few and all tokens, and lengths outside 0 .. N; what lies behind is
    never read."""
    u = util()
    lengths = [0, 1, 2, 3, 64, 65, 99, 100, 1000, -5]
    p = u.conv_problem(10, 100, 24, W, dtype, 3, lengths=lengths)
    want = la.la_forward_conv(p["x"], p["weight"], p["bias"], S0=p["S0"], return_state=True, lengths=p["lengths"])
    u.check_conv(p)
    for b, n in enumerate(lengths):
        p["x"][b, max(0, n):] = float("nan")
        p["dy"][b, max(0, n):] = float("inf")
    got = la.la_forward_conv(p["x"], p["weight"], p["bias"], S0=p["S0"], return_state=True, lengths=p["lengths"])
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    grads = la.la_backward_conv(p["dy"], p["x"], p["weight"], p["bias"], S0=p["S0"], dS_out=p["dS_out"],
                                lengths=p["lengths"])
    assert all(torch.isfinite(g).all() for g in grads)


@pytest.mark.parametrize("activation", ["silu", "sigmoid"])
@pytest.mark.parametrize("W", [2, 3, 4])
def test_infinite_last_token(W, activation):
    """What a row's last token is does not reach behind it, nor other rows and channels."""
    u = util()
    lengths = [1, 2, 3, 5, 8, 33, 64, 70]
    p = u.conv_problem(8, 70, 24, W, F32, 13, lengths=lengths)
    for b, n in enumerate(lengths):
        p["x"][b, n - 1, 0] = float("inf")
    y, _ = la.la_forward_conv(p["x"], p["weight"], p["bias"], activation=activation, S0=p["S0"], lengths=p["lengths"])
    dx, dw, db, dS0 = la.la_backward_conv(p["dy"], p["x"], p["weight"], p["bias"], activation=activation, S0=p["S0"],
                                          dS_out=p["dS_out"], lengths=p["lengths"])
    for b, n in enumerate(lengths):
        assert not y[b, n:].any() and not dx[b, n:].any()
    assert all(torch.isfinite(g).all() for g in (y[..., 1:], dx[..., 1:], dw[1:], db[1:], dS0[..., 1:]))


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("slices", [8, 3, 2, 4])
def test_strides(slices, dtype):
    """Slices of wider rows, on and off 16-byte boundaries; tokens out of a longer tensor;
    tokens in another order; one row for all (stride 0)."""
    u = util()
    p = u.conv_problem(2, 41, 32, 4, dtype, 5, slices=slices)
    assert not p["x"].is_contiguous()
    u.check_conv(p)
    p["x"] = torch.cat([p["x"]] * 3, 1)[:, 20:61]
    u.check_conv(p)
    p["x"] = p["x"].transpose(0, 1).contiguous().transpose(0, 1)
    u.check_conv(p)
    p["x"] = p["x"][:, :1].expand(-1, 41, -1)
    u.check_conv(p)


@pytest.mark.parametrize("dtype,C", [(F32, 24), (F32, 5), (BF, 24), (BF, 5)])
@pytest.mark.parametrize("W", [2, 3, 4])
def test_prompt_then_steps(W, dtype, C):
    """A prompt in two pieces and then token by token gives what one call gives, and the
    window is moved in place."""
    u = util()
    p = u.conv_problem(3, 29, C, W, dtype, 7)
    y, S = la.la_forward_conv(p["x"], p["weight"], p["bias"], S0=p["S0"], return_state=True)
    win = p["S0"].clone()
    y1, got = la.la_forward_conv(p["x"][:, :2], p["weight"], p["bias"], S0=win, S_out=win)
    assert got is win
    y2, _ = la.la_forward_conv(p["x"][:, 2:20], p["weight"], p["bias"], S0=win, S_out=win)
    rest = [la.la_decode_step_conv(win, p["x"][:, t], p["weight"], p["bias"]) for t in range(20, 29)]
    assert torch.equal(torch.cat([y1, y2, torch.stack(rest, 1)], 1), y) and torch.equal(win, S)


def test_far_sums():
    """Sums of +-1e4 saturate without a NaN; the slope keeps its digits where 1 - sigmoid
    would have none."""
    u = util()
    x = torch.tensor([-1e4, -60.0, -20.0, 14.0, 17.0, 30.0, 1e4], device="cuda").view(1, 7, 1).repeat(1, 1, 4)
    w = torch.zeros(4, 2, device="cuda")
    w[:, 1] = 1
    dy = torch.ones_like(x)
    for act in ("silu", "sigmoid"):
        y, _ = la.la_forward_conv(x, w, activation=act)
        dx = la.la_backward_conv(dy, x, w, activation=act)[0]
        v, s = ssm.act(to_np(x), act)
        # the exponential is off by 2 + 1.16 |u| of 2^-23 and zero under 2^-126
        tol = (8 + 1.5 * np.abs(to_np(x))) * 2.0 ** -23
        assert np.all(np.abs(to_np(y) - v) <= tol * np.abs(v) + 2.0 ** -110)
        assert np.all(np.abs(to_np(dx) - s) <= tol * np.abs(s) + 2.0 ** -110)


@pytest.mark.parametrize("dtype", [F32, BF])
def test_long_rows(dtype):
    """Several runs for each thread of the gradient and parts of many blocks; twice the same
    bits.  Sums of 3 * 5000 tokens: fp32 over at most a few hundred terms in a row."""
    u = util()
    p = u.conv_problem(3, 5003, 264, 4, dtype, 9, lengths=[5003, 4001, 17])
    u.check_conv(p)
    run = lambda **k: la.la_backward_conv(p["dy"], p["x"], p["weight"], p["bias"], S0=p["S0"],  # noqa: E731
                                          dS_out=p["dS_out"], lengths=p["lengths"], **k)
    need = la.la_conv_backward_workspace_size(3, 5003, 264, 4, dtype)
    ws = torch.randint(0, 256, (need + 512,), dtype=torch.uint8, device="cuda")
    tail = ws[need:].clone()
    assert all(torch.equal(a, b) for a, b in zip(run(), run(workspace=ws[:need])))
    assert torch.equal(ws[need:], tail)


def test_no_tokens():
    u = util()
    p = u.conv_problem(2, 0, 16, 4, BF, 2)
    y, S = la.la_forward_conv(p["x"], p["weight"], p["bias"], S0=p["S0"], return_state=True)
    assert y.shape == (2, 0, 16) and torch.equal(S, p["S0"])
    dx, dw, db, dS0 = la.la_backward_conv(p["dy"], p["x"], p["weight"], p["bias"], S0=p["S0"], dS_out=p["dS_out"])
    assert dx.shape == (2, 0, 16) and not dw.any() and not db.any() and torch.equal(dS0, p["dS_out"])
    _, S = la.la_forward_conv(p["x"], p["weight"], return_state=True)
    assert not S.any()


def test_graph_and_stream():
    u = util()
    p = u.conv_problem(2, 300, 64, 4, BF, 6, heads=2)
    fwd = lambda **k: la.la_forward_conv(p["x"], p["weight"], p["bias"], heads=2, return_state=True, **k)  # noqa: E731
    bwd = lambda **k: la.la_backward_conv(p["dy"], p["x"], p["weight"], p["bias"], S0=p["S0"], **k)  # noqa: E731
    want = (*fwd(), *bwd())
    side = torch.cuda.Stream()
    got = (*fwd(stream=side), *bwd(stream=side))
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = (*fwd(), *bwd())
    for _ in range(2):
        for t in got:
            t.zero_()
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_refusals():
    u = util()
    p = u.conv_problem(2, 6, 16, 4, F32, 8)
    x, w, b = p["x"], p["weight"], p["bias"]
    bad = [lambda: la.la_forward_conv(x, w.bfloat16(), b), lambda: la.la_forward_conv(x, w[:8], b),
           lambda: la.la_forward_conv(x, w, b, y=x), lambda: la.la_forward_conv(x, w, b, heads=3),
           lambda: la.la_forward_conv(x.transpose(1, 2).contiguous().transpose(1, 2), w, b),
           lambda: la.la_forward_conv(x, w, b, S0=p["S0"].bfloat16()),
           lambda: la.la_forward_conv(x, w, b, S0=p["S0"][:, :2]),
           lambda: la.la_forward_conv(x, w, b, lengths=torch.ones(2, dtype=torch.int64, device="cuda")),
           lambda: la.la_forward_conv(x, w, b, lengths=torch.ones(3, dtype=torch.int32, device="cuda")),
           lambda: la.la_forward_conv(x, w, b, lengths=torch.ones(2, dtype=torch.int32)),
           lambda: la.la_forward_conv(x.half(), w, b), lambda: la.la_backward_conv(p["dy"][:, :5], x, w, b),
           lambda: la.la_forward_conv(x, torch.zeros(16, 5, device="cuda"), b),
           lambda: la.la_decode_step_conv(p["S0"][:, :2], x[:, 0], w, b)]
    for i, f in enumerate(bad):
        with pytest.raises((ValueError, TypeError, la.LinAttnError)):
            f()
            pytest.fail(str(i))


def test_offsets_past_32_bits():
    """More than 2^31 elements: equal batch rows have equal results, those of a call of its own."""
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < (40 << 30):
        pytest.skip("needs 40 GB of device memory")
    B, N, C = 65, 8200, 4096
    g = torch.Generator(device="cuda").manual_seed(13)
    x1, dy1 = (torch.randn((1, N, C), generator=g, device="cuda").bfloat16() for _ in range(2))
    w, b = torch.randn((C, 4), generator=g, device="cuda"), torch.randn((C,), generator=g, device="cuda")
    x, dy = (t.expand(B, -1, -1).contiguous() for t in (x1, dy1))
    assert x.numel() > 2 ** 31
    y, y1 = la.la_forward_conv(x, w, b)[0], la.la_forward_conv(x1, w, b)[0]
    assert torch.equal(y, y1.expand_as(y))
    del y
    dx, dx1 = la.la_backward_conv(dy, x, w, b)[0], la.la_backward_conv(dy1, x1, w, b)[0]
    assert torch.equal(dx, dx1.expand_as(dx))
