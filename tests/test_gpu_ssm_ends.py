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


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("n,G,C,slices", [(8, 1, 20, 0), (16, 1, 20, 3), (16, 2, 36, 2), (32, 2, 24, 0), (64, 1, 33, 4),
                                          (16, 1, 131, 0), (64, 1, 16, 8)])
def test_whole_rows(n, G, C, slices, dtype):
    """So many rows that none is cut: several tiles of tokens each, ragged, on and off the boundaries of
    wide copies, the state continued in place."""
    u = util()
    B, N = 400, 45
    gen = torch.Generator().manual_seed(n + C)
    lengths = torch.randint(0, N + 1, (B,), generator=gen).tolist()
    lengths[:6] = [0, 1, 8, 16, 17, N]
    assert la.la_ssm_workspace_size(B, N, C, G, n, dtype) == 0
    p = u.ssm_problem(B, N, C, n, G, dtype, 19, lengths=lengths, slices=slices)
    u.check_ssm(p, grad=False)
    pos, kw = u.ssm_args(p)
    want = la.la_forward_ssm(*pos, **kw, S0=p["S0"], return_state=True, lengths=p["lengths"])
    S = p["S0"].clone()
    got = la.la_forward_ssm(*pos, **kw, S0=S, S_out=S, lengths=p["lengths"])
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("n", [8, 16, 32, 64])
def test_cut_rows_continued_in_place(n, dtype):
    """Ragged rows cut into segments, the state and the window in the places of the ones before: the
    same bits as in places of their own."""
    u = util()
    p = u.ssm_problem(5, 300, 24, n, 1, dtype, 21, lengths=[300, 0, 1, 150, 299])
    assert la.la_ssm_workspace_size(5, 300, 24, 1, n, dtype) > 0
    u.check_ssm(p, grad=False)
    pos, kw = u.ssm_args(p)
    want = la.la_forward_ssm(*pos, **kw, S0=p["S0"], return_state=True, lengths=p["lengths"])
    S = p["S0"].clone()
    assert all(torch.equal(a, b) for a, b in zip(la.la_forward_ssm(*pos, **kw, S0=S, S_out=S, lengths=p["lengths"]), want))
    c = u.conv_problem(5, 300, 24, 4, dtype, 21, lengths=[300, 0, 1, 150, 299])
    want = la.la_forward_conv(c["x"], c["weight"], c["bias"], S0=c["S0"], return_state=True, lengths=c["lengths"])
    W = c["S0"].clone()
    got = la.la_forward_conv(c["x"], c["weight"], c["bias"], S0=W, S_out=W, lengths=c["lengths"])
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_calls_at_once_on_two_streams():
    """Forwards and gradients of two problems on two streams, issued in turn: the bits of calls
    alone."""
    u = util()
    probs = [(u.ssm_problem(2, 500, 40, 16, 1, BF, 22 + i), u.conv_problem(2, 500, 40, 4, BF, 22 + i)) for i in range(2)]

    def run(p, c, **k):
        pos, kw = u.ssm_args(p)
        return (*la.la_forward_ssm(*pos, **kw, S0=p["S0"], return_state=True, **k),
                *la.la_backward_ssm(p["dout"], *pos, **kw, S0=p["S0"], dS_out=p["dS_out"], **k),
                la.la_forward_conv(c["x"], c["weight"], c["bias"], **k)[0],
                *la.la_backward_conv(c["dy"], c["x"], c["weight"], c["bias"], S0=c["S0"], **k))

    want = [run(*pr) for pr in probs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in probs]
    got = [[run(*pr, stream=s) for pr, s in zip(probs, streams)] for _ in range(4)]
    torch.cuda.synchronize()
    for again in got:
        for g, w in zip(again, want):
            assert all(torch.equal(a, b) for a, b in zip(g, w))
