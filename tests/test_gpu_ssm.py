"""The selective scan on the GPU against the fp64 recurrence (tolerances: ssm_util)."""
import numpy as np
import pytest
import torch

from gpu_util import to_np
from oracle import delta as delta_oracle
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
@pytest.mark.parametrize("n", [8, 16, 32, 64])
@pytest.mark.parametrize("B,N,C", [(1, 1, 1), (2, 2, 8), (1, 33, 40), (2, 67, 131), (1, 200, 16)])
def test_sizes(B, N, C, n, dtype):
    u = util()
    u.check_ssm(u.ssm_problem(B, N, C, n, 1, dtype, N + n))


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("n,G,C", [(16, 2, 32), (16, 3, 15), (8, 4, 1200), (32, 2, 180), (64, 5, 40), (16, 6, 6)])
def test_groups(n, G, C, dtype):
    """Groups smaller and larger than a block's channels."""
    u = util()
    u.check_ssm(u.ssm_problem(2, 45, C, n, G, dtype, C))


@pytest.mark.parametrize("gate", [True, False])
@pytest.mark.parametrize("extras", [True, False])
@pytest.mark.parametrize("state", [True, False])
def test_options(gate, extras, state):
    u = util()
    u.check_ssm(u.ssm_problem(2, 70, 24, 16, 1, F32, 1, gate=gate, extras=extras, state=state))


def test_steps_as_given():
    """Without the softplus a step may be zero (the token leaves no trace) or large."""
    u = util()
    p = u.ssm_problem(2, 50, 16, 16, 1, F32, 2, extras=False)
    p["delta"] = p["delta"].abs() * 0.5
    p["delta"][:, 10:20] = 0
    u.check_ssm(p, softplus=False)
    p["delta"][:, 30] = 60.0  # a reset: exp(-60 A) is nothing
    u.check_ssm(p, softplus=False)


def test_zero_steps_leave_the_state():
    u = util()
    p = u.ssm_problem(2, 100, 40, 16, 1, F32, 3, extras=False)
    p["delta"].zero_()
    pos, kw = u.ssm_args(p)
    _, S = la.la_forward_ssm(*pos, **kw, softplus=False, S0=p["S0"], return_state=True)
    assert torch.equal(S, p["S0"])
    S = p["S0"].clone()
    la.la_decode_step_ssm(S, p["x"][:, 0], p["delta"][:, 0], p["A"], p["Bm"][:, 0], p["Cm"][:, 0], softplus=False)
    assert torch.equal(S, p["S0"])


def test_far_steps():
    """delta + bias from -80 (no step) to 40 (the step itself): every digit of small steps, no
    overflow of large ones."""
    u = util()
    p = u.ssm_problem(1, 60, 16, 16, 1, F32, 4, extras=False)
    p["delta"] = torch.linspace(-80, 40, 60, device="cuda").view(1, 60, 1).repeat(1, 1, 16)
    u.check_ssm(p)
    S = torch.zeros(60, 4, 8, device="cuda")
    raw = torch.linspace(-80, 40, 60, device="cuda").view(60, 1).repeat(1, 4)
    one = torch.ones(60, 1, 8, device="cuda")
    la.la_decode_step_ssm(S, torch.ones(60, 4, device="cuda"), raw, torch.zeros(4, 8, device="cuda"), one, one)
    want = ssm.softplus(to_np(raw))[0]
    # the exponential of u is off by 2 + 1.16 |u| of 2^-23, the rest by a few
    assert np.all(np.abs(to_np(S)[..., 0] - want) <= (8 + 1.5 * np.abs(to_np(raw))) * 2.0 ** -23 * want)


def test_long_memory():
    """Steps of 1e-4 to 1e-3 with rates of 1: states that remember every token.  A state adds up
    the mean error of at most N = 3000 decays, 0.29 * 2^-24 each: 5.2e-5 at most."""
    u = util()
    p = u.ssm_problem(1, 3000, 16, 8, 1, F32, 5, low=1e-4)
    p["delta_bias"] -= 2
    u.check_ssm(p, tol=5.2e-5)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("n", [8, 16, 32, 64])
def test_lengths(n, dtype):
    """Rows of no, one, few and all tokens, lengths outside 0 .. N; what lies behind is never read."""
    u = util()
    lengths = [0, 1, 3, 8, 31, 32, 33, 64, 99, 100, 1000, -5]
    p = u.ssm_problem(12, 100, 20, n, 1, dtype, 6, lengths=lengths)
    pos, kw = u.ssm_args(p)
    run = lambda: la.la_forward_ssm(*pos, **kw, S0=p["S0"], return_state=True, lengths=p["lengths"])  # noqa: E731
    back = lambda: la.la_backward_ssm(p["dout"], *pos, **kw, S0=p["S0"], dS_out=p["dS_out"],  # noqa: E731
                                      lengths=p["lengths"])
    u.check_ssm(p)
    want = (*run(), *back())
    for b, m in enumerate(lengths):
        for name in ("x", "delta", "z", "dout", "Bm", "Cm"):
            p[name][b, max(0, m):] = float("nan")
    assert all(torch.equal(a, b) for a, b in zip((*run(), *back()), want))


@pytest.mark.parametrize("n", [8, 16, 32, 64])
def test_infinite_last_token(n):
    """A state that the row's last token made infinite does not reach behind it."""
    u = util()
    lengths = [1, 2, 3, 5, 30, 33, 67, 70]
    p = u.ssm_problem(8, 70, 20, n, 1, F32, 16, lengths=lengths)
    for b, m in enumerate(lengths):
        p["x"][b, m - 1] = float("inf")
    pos, kw = u.ssm_args(p)
    out, _ = la.la_forward_ssm(*pos, **kw, S0=p["S0"], lengths=p["lengths"])
    g = dict(zip(u.LEAVES, la.la_backward_ssm(p["dout"], *pos, **kw, S0=p["S0"], dS_out=p["dS_out"],
                                              lengths=p["lengths"])))
    for b, m in enumerate(lengths):
        assert not out[b, m:].any()
        for name in ("x", "delta", "z", "Bm", "Cm"):
            assert not g[name][b, m:].any(), (name, m)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("slices,n", [(8, 16), (3, 16), (2, 16), (8, 8), (6, 8), (5, 32), (4, 32), (16, 64), (2, 64)])
def test_strides(slices, n, dtype):
    """Slices of wider rows on boundaries of 16, 8, 4 and 2 bytes, in pieces of a longer sequence."""
    u = util()
    p = u.ssm_problem(2, 41, 32, n, 1, dtype, 7, slices=slices)
    assert not p["x"].is_contiguous() and not p["Cm"].is_contiguous()
    u.check_ssm(p)
    q = dict(p)
    for name in ("x", "delta", "z", "dout", "Bm", "Cm"):
        q[name] = torch.cat([p[name]] * 2, 1)[:, 5:46]
    u.check_ssm(q)
    for name in ("x", "delta", "z", "dout", "Bm", "Cm"):
        q[name] = p[name].transpose(0, 1).contiguous().transpose(0, 1)
    u.check_ssm(q)


def test_one_row_for_all():
    """Broadcast inputs (stride 0): the gradient is that of every row."""
    u = util()
    p = u.ssm_problem(3, 20, 16, 16, 1, F32, 8)
    for name in ("x", "delta", "z", "Bm", "Cm"):
        p[name] = p[name][:1].expand(3, *p[name].shape[1:])
    u.check_ssm(p)


@pytest.mark.parametrize("dtype,C,n,G", [(F32, 24, 16, 1), (BF, 24, 16, 2), (BF, 5, 8, 1), (F32, 33, 32, 1),
                                         (BF, 18, 64, 1)])
def test_prompt_then_steps(dtype, C, n, G):
    """A prompt in two pieces and then token by token: the outputs of one call, states in place."""
    u = util()
    p = u.ssm_problem(3, 61, C, n, G, dtype, 9)
    pos, kw = u.ssm_args(p)
    ref, r_S = ssm_oracle_pair(u, p)
    S = p["S0"].clone()

    def piece(lo, hi):
        cut = lambda t: t[:, lo:hi]  # noqa: E731
        out, got = la.la_forward_ssm(cut(p["x"]), cut(p["delta"]), p["A"], cut(p["Bm"]), cut(p["Cm"]), D=p["D"],
                                     z=cut(p["z"]), delta_bias=p["delta_bias"], S0=S, S_out=S)
        assert got is S
        return out

    outs = [piece(0, 33), piece(33, 50)]
    for t in range(50, 61):
        outs.append(la.la_decode_step_ssm(S, p["x"][:, t], p["delta"][:, t], p["A"], p["Bm"][:, t], p["Cm"][:, t],
                                          D=p["D"], z=p["z"][:, t], delta_bias=p["delta_bias"])[:, None])
    u.near(torch.cat(outs, 1), ref, "out")
    u.near(S, r_S, "S")


def ssm_oracle_pair(u, p):
    return u.ssm_oracle(p)


@pytest.mark.parametrize("B,C,n,G,dtype", [(1, 1, 8, 1, F32), (5, 250, 32, 2, F32), (37, 96, 16, 1, BF),
                                           (3, 77, 64, 7, BF), (200, 64, 16, 1, BF)])
def test_step(B, C, n, G, dtype):
    u = util()
    p = u.ssm_problem(B, 1, C, n, G, dtype, 10)
    S = p["S0"].clone()
    out = la.la_decode_step_ssm(S, p["x"][:, 0], p["delta"][:, 0], p["A"], p["Bm"][:, 0], p["Cm"][:, 0], D=p["D"],
                                z=p["z"][:, 0], delta_bias=p["delta_bias"])
    ref, r_S = u.ssm_oracle(p)
    u.near(out, ref[:, 0], "out")
    u.near(S, r_S, "S")


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("B,C,n,G,slices", [(203, 128, 16, 1, 0), (401, 129, 8, 3, 0), (37, 160, 64, 2, 0), (82, 130, 32, 1, 3),
                                            (206, 98, 16, 2, 4)])
def test_step_of_many_rows(B, C, n, G, slices, dtype):
    """Several rows a thread, batches that do not divide by them, B and C on and off the boundaries
    of their loads."""
    u = util()
    p = u.ssm_problem(B, 1, C, n, G, dtype, 15, slices=slices)
    S = p["S0"].clone()
    out = la.la_decode_step_ssm(S, p["x"][:, 0], p["delta"][:, 0], p["A"], p["Bm"][:, 0], p["Cm"][:, 0], D=p["D"],
                                z=p["z"][:, 0], delta_bias=p["delta_bias"])
    ref, r_S = u.ssm_oracle(p)
    u.near(out, ref[:, 0], "out")
    u.near(S, r_S, "S")


def test_captured_steps():
    """A captured step moves window and state on at every replay, as eager calls do."""
    u = util()
    p, c = u.ssm_problem(3, 1, 64, 16, 1, BF, 16), u.conv_problem(3, 1, 64, 4, BF, 16)
    step = [p[k][:, 0] for k in ("delta", "A", "Bm", "Cm")]
    step[1] = p["A"]

    def one(win, S):
        x = la.la_decode_step_conv(win, c["x"][:, 0], c["weight"], c["bias"])
        return la.la_decode_step_ssm(S, x, *step, D=p["D"], z=p["z"][:, 0], delta_bias=p["delta_bias"])

    win, S = c["S0"].clone(), p["S0"].clone()
    want = [one(win, S).clone() for _ in range(3)]
    win2, S2 = c["S0"].clone(), p["S0"].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = one(win2, S2)
    for k in range(3):
        graph.replay()
        assert torch.equal(out, want[k]), k
    assert torch.equal(win, win2) and torch.equal(S, S2)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("B,N,C,n", [(400, 20, 16, 16), (1, 1500, 200, 16), (2, 1111, 24, 8), (1, 700, 520, 64), (40, 40, 512, 16)])
def test_segments(B, N, C, n, dtype):
    """Few long rows (segments and their join) and many short ones, twice the same bits; scratch
    of any content, none of it written behind its end.  N = 1500: the mean error of a decay
    adds up to 2.6e-5 at most."""
    u = util()
    p = u.ssm_problem(B, N, C, n, 1, dtype, 11)
    u.check_ssm(p, tol=max(1e-5, 1.75e-8 * N))
    pos, kw = u.ssm_args(p)
    for need, run in (
            (la.la_ssm_workspace_size(B, N, C, 1, n, dtype),
             lambda **k: la.la_forward_ssm(*pos, **kw, S0=p["S0"], return_state=True, **k)),
            (la.la_ssm_backward_workspace_size(B, N, C, 1, n, dtype),
             lambda **k: la.la_backward_ssm(p["dout"], *pos, **kw, S0=p["S0"], dS_out=p["dS_out"], **k))):
        ws = torch.randint(0, 256, (need + 512,), dtype=torch.uint8, device="cuda")
        tail = ws[need:].clone()
        assert all(torch.equal(a, b) for a, b in zip(run(), run(workspace=ws[:need])))
        assert torch.equal(ws[need:], tail)


def test_gradients_as_differences():
    """The outputs are linear in x, Bm, Cm and D and in S0: half the difference of two forwards a step
    of one apart is the gradient itself, to the rounding of the forwards' sums (1e-5 of the sum of
    their terms' sizes)."""
    u = util()
    p = u.ssm_problem(2, 90, 40, 16, 1, F32, 12)
    pos, kw = u.ssm_args(p)
    grads = dict(zip(u.LEAVES, la.la_backward_ssm(p["dout"], *pos, **kw, S0=p["S0"], dS_out=p["dS_out"])))
    g = torch.Generator(device="cuda").manual_seed(1)
    for name in ("x", "Bm", "Cm", "D", "S0"):
        v = torch.randn(p[name].shape, generator=g, device="cuda")
        loss, size = [], 0.0
        for sign in (1, -1):
            q = dict(p, **{name: p[name] + sign * v})
            pos, kw = u.ssm_args(q)
            out, S = la.la_forward_ssm(*pos, **kw, S0=q["S0"], return_state=True)
            terms = (out.double() * p["dout"]).sum() + (S.double() * p["dS_out"]).sum()
            size = max(size, float((out.double() * p["dout"]).abs().sum() + (S.double() * p["dS_out"]).abs().sum()))
            loss.append(float(terms))
        want = float((grads[name].double() * v).sum())
        assert abs((loss[0] - loss[1]) / 2 - want) <= 1e-5 * size, (name, loss, want)


def test_strong_decays():
    """Rates of 1000 with steps near 0.1: nothing is left of a state after a token; dA is then
    tiny and keeps its digits (exp(-x) is off by about x 2^-24, here x up to 40)."""
    u = util()
    p = u.ssm_problem(1, 40, 16, 16, 1, F32, 14, gate=False)
    p["A"] = -torch.linspace(1, 1000, 256, device="cuda").view(16, 16)
    u.check_ssm(p)


def test_no_tokens():
    u = util()
    p = u.ssm_problem(2, 0, 16, 16, 1, BF, 2)
    pos, kw = u.ssm_args(p)
    out, S = la.la_forward_ssm(*pos, **kw, S0=p["S0"], return_state=True)
    assert out.shape == (2, 0, 16) and torch.equal(S, p["S0"])
    g = dict(zip(u.LEAVES, la.la_backward_ssm(p["dout"], *pos, **kw, S0=p["S0"], dS_out=p["dS_out"])))
    assert torch.equal(g["S0"], p["dS_out"]) and not any(g[k].any() for k in ("A", "D", "delta_bias"))
    _, S = la.la_forward_ssm(*pos, return_state=True)
    assert not S.any()


def test_graph_and_stream():
    u = util()
    p = u.ssm_problem(1, 700, 64, 16, 1, BF, 6)
    pos, kw = u.ssm_args(p)
    fwd = lambda **k: la.la_forward_ssm(*pos, **kw, S0=p["S0"], return_state=True, **k)  # noqa: E731
    bwd = lambda **k: la.la_backward_ssm(p["dout"], *pos, **kw, S0=p["S0"], **k)  # noqa: E731
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
    p = u.ssm_problem(2, 6, 16, 16, 1, F32, 8)
    x, d, A, Bm, Cm = u.ssm_args(p)[0]
    S = torch.zeros(2, 16, 16, device="cuda")
    bad = [lambda: la.la_forward_ssm(x, d, A.bfloat16(), Bm, Cm), lambda: la.la_forward_ssm(x, d, A[:8], Bm, Cm),
           lambda: la.la_forward_ssm(x, d, A, Bm, Cm, x), lambda: la.la_forward_ssm(x, d, A, Bm, Cm, d),
           lambda: la.la_forward_ssm(x, d, A, Bm, Cm, p["z"], z=p["z"]),
           lambda: la.la_forward_ssm(x, d.bfloat16(), A, Bm, Cm), lambda: la.la_forward_ssm(x, d[:, :5], A, Bm, Cm),
           lambda: la.la_forward_ssm(x, d, A, Bm[:, :, 0], Cm[:, :, 0]),
           lambda: la.la_forward_ssm(x, d, A[:, :4].contiguous(), Bm[..., :4].contiguous(), Cm[..., :4].contiguous()),
           lambda: la.la_forward_ssm(x, d, A, Bm.expand(-1, -1, 3, -1), Cm.expand(-1, -1, 3, -1)),
           lambda: la.la_forward_ssm(x, d, A, Bm.transpose(1, 3).contiguous().transpose(1, 3), Cm),
           lambda: la.la_forward_ssm(x, d, A, Bm, Cm, S0=S.bfloat16()),
           lambda: la.la_forward_ssm(x, d, A, Bm, Cm, lengths=torch.ones(2, device="cuda")),
           lambda: la.la_decode_step_ssm(S[:1], x[:, 0], d[:, 0], A, Bm[:, 0], Cm[:, 0]),
           lambda: la.la_decode_step_ssm(S, x, d, A, Bm, Cm),
           lambda: la.la_backward_ssm(p["dout"][:, :3], x, d, A, Bm, Cm)]
    for i, f in enumerate(bad):
        with pytest.raises((ValueError, TypeError, la.LinAttnError)):
            f()
            pytest.fail(str(i))


@pytest.mark.parametrize("dtype", [F32, BF])
def test_a_layer(dtype):
    """A layer as it would be used: one projection's slices through the convolution and the scan, in
    two ragged prompts and then a token each; forwards against the oracle on the inputs that each
    call was given, and the gradients of the pair by the chain rule."""
    u = util()
    B, N, C, n, W = 2, 45, 48, 16, 4
    g = torch.Generator().manual_seed(77)
    m = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    xz, dbc = m(B, N, 2 * C).to(dtype).cuda(), m(B, N, 8 + 2 * n).to(dtype).cuda()
    w, b, A = m(C, W).cuda(), m(C).cuda(), -torch.exp(m(C, n)).cuda()
    D, lengths = m(C).cuda(), torch.tensor([45, 21], dtype=torch.int32, device="cuda")
    raw = (m(B, N, C) - 3).to(dtype).cuda()
    x, win = la.la_forward_conv(xz[..., :C], w, b, return_state=True, lengths=lengths)
    Bm, Cm = dbc[..., 8:8 + n].unflatten(-1, (1, n)), dbc[..., 8 + n:].unflatten(-1, (1, n))
    out, S = la.la_forward_ssm(x, raw, A, Bm, Cm, D=D, z=xz[..., C:], return_state=True, lengths=lengths)
    ry, rwin = ssm.conv(to_np(xz[..., :C]), to_np(w), to_np(b), lengths=to_np(lengths))
    u.near(x, ry, "x")
    assert np.array_equal(to_np(win), rwin)
    scan = lambda **k: ssm.scan(to_np(x), to_np(raw), to_np(A), to_np(Bm), to_np(Cm), D=to_np(D),  # noqa: E731
                                z=to_np(xz[..., C:]), lengths=to_np(lengths), **k)
    dout = m(B, N, C).to(dtype).cuda()
    ref = scan(dout=to_np(dout))
    u.near(out, ref["out"], "out")
    u.near(S, ref["S"], "S")
    grads = la.la_backward_ssm(dout, x, raw, A, Bm, Cm, D=D, z=xz[..., C:], lengths=lengths)
    dx, dw, db, _ = la.la_backward_conv(grads[0], xz[..., :C], w, b, lengths=lengths)
    _, _, rdx, rdw, rdb, _ = ssm.conv(to_np(xz[..., :C]), to_np(w), to_np(b), lengths=to_np(lengths),
                                      dy=to_np(grads[0]))
    for got, want, name in ((grads[0], ref["x"], "dx"), (grads[2], ref["A"], "dA"), (dx, rdx, "conv dx"),
                            (dw, rdw, "dw"), (db, rdb, "db")):
        u.near(got, want, name)
    # one more token for each row
    new = m(B, 2 * C).to(dtype).cuda()
    x1 = la.la_decode_step_conv(win, new[:, :C], w, b)
    S_before, one = S.clone(), dbc[:, 3]
    o1 = la.la_decode_step_ssm(S, x1, raw[:, 3], A, one[:, 8:8 + n].unflatten(-1, (1, n)),
                               one[:, 8 + n:].unflatten(-1, (1, n)), D=D, z=new[:, C:])
    r1, rS = ssm.scan(to_np(x1)[:, None], to_np(raw[:, 3:4]), to_np(A), to_np(Bm[:, 3:4]), to_np(Cm[:, 3:4]), D=to_np(D),
                      z=to_np(new[:, C:])[:, None], S0=to_np(S_before))
    u.near(o1, r1[:, 0], "step")
    u.near(S, rS, "S after the step")


def test_conv_in_front_of_the_delta_rule():
    """Queries, keys and values out of one projection, convolved and handed head-major to the delta
    rule, against its oracle on the same heads."""
    B, N, H, d = 1, 70, 2, 32
    g = torch.Generator().manual_seed(5)
    qkv = torch.randn((B, N, 3 * H * d), generator=g).cuda()
    w = torch.randn((3, H * d, 4), generator=g).cuda()
    q, k, v = (la.la_forward_conv(qkv[..., i * H * d:(i + 1) * H * d], w[i], heads=H)[0] for i in range(3))
    beta = torch.sigmoid(torch.randn((B, H, N), generator=g)).cuda()
    out, S = la.la_forward_delta(q, k, v, beta, return_state=True)
    r, rS = delta_oracle.forward(*map(to_np, (q, k, v, beta)), scale=d ** -0.5)
    util().near(out, r, "out")
    util().near(S, rS, "S")


def test_offsets_past_32_bits():
    """More than 2^31 elements: equal batch rows have equal results, those of a call of its own."""
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < (120 << 30):
        pytest.skip("needs 120 GB of device memory")
    B, N, C, n = 66, 8000, 4096, 8
    g = torch.Generator(device="cuda").manual_seed(13)
    m = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()  # noqa: E731
    one = dict(x=m(1, N, C), delta=m(1, N, C) - 3, Bm=m(1, N, 1, n), Cm=m(1, N, 1, n), dout=m(1, N, C))
    A = -torch.rand((C, n), generator=g, device="cuda") - 0.5
    many = {k: t.expand(B, *t.shape[1:]).contiguous() for k, t in one.items()}
    assert many["x"].numel() > 2 ** 31
    run = lambda p: la.la_forward_ssm(p["x"], p["delta"], A, p["Bm"], p["Cm"])[0]  # noqa: E731
    out, out1 = run(many), run(one)
    # the single row is cut into segments, the 66 are not: bf16 results one rounding apart at most
    assert torch.equal(out, out[:1].expand_as(out))
    assert (out[0].float() - out1[0].float()).abs().max() <= 2.0 ** -7 * out1.float().abs().max()
    del out
    back = lambda p: la.la_backward_ssm(p["dout"], p["x"], p["delta"], A, p["Bm"], p["Cm"])  # noqa: E731
    got, want = back(many), back(one)
    for i in (0, 1, 3, 4):
        assert torch.equal(got[i], want[i].expand_as(got[i])), i
