"""The gated delta rule on the GPU against the fp64 recurrence.

Tolerances.  A rounding to bf16 is off by at most h = 2^-8 of the value.
 - fp32 results (states, gate gradients, and everything with fp32 inputs):
   1e-5 of the tensor's 2-norm and of its largest entry, the library's bound
   for fp32.  With bf16 inputs an fp32 operand of a tensor-core product is the
   sum of two bf16 parts, off by at most h^2 = 1.5e-5 per term and by about a
   fifth of that in the mean over independent terms.
 - bf16 outputs: the result is rounded once (h |o|), and each of the two
   products that make it up may have one operand rounded to bf16 besides its
   exact one or two of them rounded: at most 2 h of the sum of the terms'
   absolute values (the oracle's `mag`), per element.
 - 2-norm of bf16 results: independent roundings of the result and of two
   operands are each at most h / sqrt(3) in the mean: sqrt(3) h / sqrt(3) = h;
   with a factor of two for rounding errors that are not independent, 2 h.
 - largest entry of bf16 gradients: h of the result and twice h of operands,
   within 4 h of the largest entry.
"""
import numpy as np
import pytest
import torch

from gpu_util import to_np
from oracle import delta

pytestmark = pytest.mark.gpu

la = pytest.importorskip("kernelised_causal_linear_gb300")

H8 = 2.0 ** -8
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.fail("GPU test run without a CUDA device")
    yield
    assert la.la_get_device_status() == 0


def problem(B, H, Hk, N, d, dv, dtype, seed=0, gated=True, state=True, l2=True):
    g = torch.Generator().manual_seed(1000 + seed)
    n = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    qk = 1.0 if l2 else d ** -0.5
    p = dict(q=(n(B, Hk, N, d) * qk).to(dtype), k=(n(B, Hk, N, d) * qk).to(dtype),
             v=n(B, H, N, dv).to(dtype), beta=torch.sigmoid(n(B, H, N)),
             log_alpha=-torch.nn.functional.softplus(2 * n(B, H, N) - 2) if gated else None,
             S0=0.3 * n(B, H, d, dv) if state else None, dout=n(B, H, N, dv).to(dtype),
             dS_out=0.3 * n(B, H, d, dv) if state else None)
    return {k: None if v is None else v.cuda().contiguous() for k, v in p.items()}


def host(p, *names):
    return [None if p[n] is None else to_np(p[n]) for n in names]


INPUTS = ("q", "k", "v", "beta", "log_alpha")


def far(got, ref):
    g, r = to_np(got), np.asarray(ref)
    assert g.shape == r.shape and np.all(np.isfinite(g))
    if not g.size:
        return 0.0, 0.0
    e = g - r
    return (np.linalg.norm(e) / max(np.linalg.norm(r), 1e-30),
            np.abs(e).max() / max(np.abs(r).max(), 1e-30))


def assert_fp32(got, ref, what):
    two, most = far(got, ref)
    print(f"{what}: 2-norm {two:.2e}, largest {most:.2e}")
    assert two <= 1e-5 and most <= 1e-5, (what, two, most)


def check_forward(p, l2=True, scale=None):
    scale = p["q"].shape[-1] ** -0.5 if scale is None else scale
    out, S = la.la_forward_delta(*(p[n] for n in INPUTS), feature_map="l2" if l2 else "none",
                                 scale=scale, S0=p["S0"], return_state=True)
    ro, rS, mag = delta.forward(*host(p, *INPUTS), scale=scale, l2=l2, S0=host(p, "S0")[0],
                                magnitude=True)
    assert out.dtype == p["v"].dtype and S.dtype == F32
    assert_fp32(S, rS, "S")
    if out.dtype == F32:
        assert_fp32(out, ro, "out")
    else:
        two, _ = far(out, ro)
        print(f"out: 2-norm {two:.2e}")
        err = np.abs(to_np(out) - ro)
        assert np.all(err <= H8 * np.abs(ro) + (2 * H8 + 1e-5) * mag + 1e-30)
        assert two <= 2 * H8
    return out, S


NAMES = ("dq", "dk", "dv", "dbeta", "dlog_alpha", "dS0")


def check_backward(p, l2=True, scale=None, skip=()):
    scale = p["q"].shape[-1] ** -0.5 if scale is None else scale
    got = la.la_backward_delta(p["dout"], *(p[n] for n in INPUTS),
                               feature_map="l2" if l2 else "none", scale=scale, S0=p["S0"],
                               dS_out=p["dS_out"])
    ref = delta.backward(host(p, "dout")[0], *host(p, *INPUTS), scale=scale, l2=l2,
                         S0=host(p, "S0")[0], dS_out=host(p, "dS_out")[0])
    for name, g, r in zip(NAMES, got, ref):
        if name == "dlog_alpha" and p["log_alpha"] is None or name == "dS0" and p["S0"] is None:
            assert g is None
            continue
        if name in skip:
            assert torch.isfinite(g).all()
        elif g.dtype == F32:
            assert_fp32(g, r, name)
        else:
            two, most = far(g, r)
            print(f"{name}: 2-norm {two:.2e}, largest {most:.2e}")
            assert two <= 2 * H8 and most <= 4 * H8, (name, two, most)
    return got


DIMS = [(32, 32), (32, 64), (32, 128), (64, 32), (64, 64), (64, 128), (128, 32), (128, 64),
        (128, 128)]
LENGTHS = [1, 2, 16, 31, 33, 63, 64, 65, 128, 129, 257]


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("d,dv", DIMS)
def test_forward_dims(d, dv, dtype):
    check_forward(problem(2, 4, 2, 150, d, dv, dtype, seed=d + dv))


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("N", LENGTHS)
def test_forward_lengths(N, dtype):
    check_forward(problem(1, 3, 3, N, 64, 64, dtype, seed=N))


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("gated,state,l2", [(False, False, True), (True, False, False),
                                            (False, True, False), (True, True, True)])
def test_forward_options(gated, state, l2, dtype):
    check_forward(problem(2, 6, 1, 200, 128, 64, dtype, 7, gated, state, l2), l2, scale=0.7)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("d,dv", DIMS)
def test_backward_dims(d, dv, dtype):
    check_backward(problem(2, 4, 2, 150, d, dv, dtype, seed=3 * d + dv))


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("N", LENGTHS)
def test_backward_lengths(N, dtype):
    check_backward(problem(1, 3, 3, N, 64, 64, dtype, seed=N))


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("gated,state,l2", [(False, False, True), (True, False, False),
                                            (False, True, False), (True, True, True)])
def test_backward_options(gated, state, l2, dtype):
    check_backward(problem(2, 6, 1, 200, 128, 64, dtype, 8, gated, state, l2), l2, scale=0.7)


@pytest.mark.parametrize("dtype", [F32, BF])
def test_long_sequences(dtype):
    """Few heads over many chunks; the state has been overwritten many times."""
    p = problem(1, 2, 1, 3001, 128, 128, dtype, 9)
    check_forward(p)
    check_backward(p)


@pytest.mark.parametrize("dtype", [F32, BF])
def test_one_key_everywhere(dtype):
    """The same key at every token with beta = 1 and no decay: each chunk's
    system is as far from diagonal as it gets, and the state holds the last
    value alone."""
    p = problem(1, 2, 2, 130, 64, 64, dtype, 10, gated=False, state=False)
    p["k"][:] = p["k"][:, :, :1]
    p["beta"][:] = 1.0
    check_forward(p)
    check_backward(p)


@pytest.mark.parametrize("dtype", [F32, BF])
def test_resets_and_gates_of_every_size(dtype):
    """log_alpha from 0 over -100 to -inf, beta 0, 1 and 2, a zero key and a
    zero query under the L2 norm."""
    p = problem(1, 4, 2, 200, 64, 64, dtype, 11)
    g = torch.Generator().manual_seed(5)
    kinds = torch.tensor([0.0, -1e-4, -0.5, -20.0, -100.0, -200.0, -np.inf])
    p["log_alpha"] = kinds[torch.randint(0, 7, (1, 4, 200), generator=g)].cuda()
    p["beta"] = torch.tensor([0.0, 0.3, 1.0, 2.0])[torch.randint(0, 4, (1, 4, 200), generator=g)].cuda()
    p["k"][:, :, 17] = 0
    p["q"][:, :, 33] = 0
    check_forward(p)
    # rows of length zero: their unit vectors have slope 1/sqrt(1e-6), so dk and
    # dq there are a thousand times the others and carry the error of a row
    # that is not normalised; everything else is checked as usual
    check_backward(p, skip=("dq", "dk"))
    p = problem(1, 4, 2, 200, 64, 64, dtype, 12)
    p["log_alpha"] = kinds[torch.randint(0, 7, (1, 4, 200), generator=g)].cuda()
    p["beta"] = torch.tensor([0.0, 0.3, 1.0, 2.0])[torch.randint(0, 4, (1, 4, 200), generator=g)].cuda()
    check_backward(p)


def test_right_padding_leaves_the_state():
    """beta = 0 and log_alpha = 0 behind the last token: the final state is the
    unpadded one's, and the gradients of the padding are zero."""
    p = problem(2, 2, 2, 100, 64, 64, BF, 13)
    p["beta"][:, :, 77:] = 0
    p["log_alpha"][:, :, 77:] = 0
    _, S = check_forward(p)
    short = {n: (x[:, :, :77].contiguous() if n in INPUTS + ("dout",) else x) for n, x in p.items()}
    _, Ss = check_forward(short)
    assert_fp32(S, to_np(Ss), "S")
    p["dout"][:, :, 77:] = 0
    dq, dk, dv, db, _, _ = check_backward(p)
    for g in (dq, dk, dv):
        assert not g[:, :, 77:].any()


@pytest.mark.parametrize("dtype", [F32, BF])
def test_state_in_place_state_only_and_no_tokens(dtype):
    p = problem(2, 4, 2, 90, 64, 128, dtype, 14)
    args = [p[n] for n in INPUTS]
    out, S = la.la_forward_delta(*args, S0=p["S0"], return_state=True)
    St = p["S0"].clone()
    o2, S2 = la.la_forward_delta(*args, S0=St, S_out=St)
    assert S2 is St and torch.equal(St, S) and torch.equal(o2, out)
    none, S3 = la.la_forward_delta(None, *args[1:], S0=p["S0"])
    assert none is None and torch.equal(S3, S)
    o4, nothing = la.la_forward_delta(*args, S0=p["S0"])
    assert nothing is None and torch.equal(o4, out)
    empty = [x[:, :, :0].contiguous() for x in args]
    o5, S5 = la.la_forward_delta(*empty, S0=p["S0"], return_state=True)
    assert o5.numel() == 0 and torch.equal(S5, p["S0"])
    _, S6 = la.la_forward_delta(*empty, return_state=True)
    assert not S6.any()
    g = la.la_backward_delta(p["dout"][:, :, :0].contiguous(), *empty, S0=p["S0"], dS_out=p["dS_out"])
    assert torch.equal(g[5], p["dS_out"]) and g[0].numel() == 0


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("d,dv", DIMS)
def test_decode_step(d, dv, dtype):
    p = problem(5, 6, 3, 4, d, dv, dtype, seed=d * dv)
    S = p["S0"].clone()
    ro, rS = delta.forward(*host(p, *INPUTS), scale=d ** -0.5, S0=host(p, "S0")[0])
    for t in range(4):
        x = [p[n][:, :, t].contiguous() for n in INPUTS]
        o = la.la_decode_step_delta(S, *x)
        two, most = far(o, ro[:, :, t])
        if dtype == F32:
            assert two <= 1e-5 and most <= 1e-5
        else:
            assert np.all(np.abs(to_np(o) - ro[:, :, t]) <= H8 * np.abs(ro[:, :, t]) + 1e-5)
    assert_fp32(S, rS, "S")


def test_decode_options():
    p = problem(3, 2, 2, 1, 64, 64, F32, 15, gated=False, l2=False)
    S = p["S0"].clone()
    x = [None if p[n] is None else p[n][:, :, 0].contiguous() for n in INPUTS]
    o = la.la_decode_step_delta(S, *x, feature_map="none", scale=2.0)
    ro, rS = delta.forward(*host(p, *INPUTS), scale=2.0, l2=False, S0=host(p, "S0")[0])
    assert_fp32(o, ro[:, :, 0], "out")
    assert_fp32(S, rS, "S")


def test_decode_a_large_batch():
    """More heads than SMs, every state compared with the chunked forward's."""
    p = problem(67, 12, 4, 1, 128, 128, BF, 16)
    S = p["S0"].clone()
    o = la.la_decode_step_delta(S, *(p[n][:, :, 0].contiguous() for n in INPUTS))
    out, Sf = la.la_forward_delta(*(p[n] for n in INPUTS), S0=p["S0"], return_state=True)
    assert_fp32(S, to_np(Sf), "S")
    assert far(o, to_np(out[:, :, 0]))[0] <= 2 * H8


def test_prefill_then_decode_then_norm():
    """The operators as a layer uses them when it serves: a prompt in two
    pieces, then tokens one by one, each through norm and gate."""
    B, H, Hk, N, d = 2, 4, 2, 190, 64
    p = problem(B, H, Hk, N, d, d, BF, 17, state=False)
    ro, rS = delta.forward(*host(p, *INPUTS), scale=d ** -0.5)
    gate = torch.randn(B, N, H, d, generator=torch.Generator().manual_seed(3)).to(BF).cuda()
    w = (1 + 0.1 * torch.randn(d, generator=torch.Generator().manual_seed(4))).cuda()
    ry = delta.norm_gate(ro, to_np(gate), to_np(w))
    cut = lambda lo, hi: [p[n][:, :, lo:hi].contiguous() for n in INPUTS]  # noqa: E731
    S = None
    for lo, hi in ((0, 100), (100, 180)):
        out, S = la.la_forward_delta(*cut(lo, hi), S0=S, return_state=True)
        y = la.la_norm_gate(out, gate[:, lo:hi].contiguous(), w)
        # two roundings to bf16 on top of the forward's operands
        assert far(y, ry[:, lo:hi])[0] <= 3 * H8
    for t in range(180, N):
        o = la.la_decode_step_delta(S, *(x[:, :, 0].contiguous() for x in cut(t, t + 1)))
        y = la.la_norm_gate(o.unsqueeze(2), gate[:, t:t + 1].contiguous(), w)
        assert far(y[:, 0], ry[:, t])[0] <= 3 * H8
    assert_fp32(S, rS, "S")


@pytest.mark.parametrize("dtype", [F32, BF])
def test_training_step_through_both(dtype):
    """Forward, norm and gate, and back to q, k, v, the gates and the weight."""
    B, H, Hk, N, d, dv = 2, 4, 2, 140, 64, 64
    p = problem(B, H, Hk, N, d, dv, dtype, 18, state=False)
    gen = torch.Generator().manual_seed(6)
    gate = torch.randn(B, N, H, dv, generator=gen).to(dtype).cuda()
    dy = torch.randn(B, N, H, dv, generator=gen).to(dtype).cuda()
    w = (1 + 0.1 * torch.randn(H, dv, generator=gen)).cuda()
    out, _ = la.la_forward_delta(*(p[n] for n in INPUTS))
    dx, dgate, dw = la.la_norm_gate_backward(dy, out, gate, w)
    grads = la.la_backward_delta(dx, *(p[n] for n in INPUTS))
    ro, _ = delta.forward(*host(p, *INPUTS), scale=d ** -0.5)
    _, rdx, rdgate, rdw = delta.norm_gate(ro, to_np(gate), to_np(w), dy=to_np(dy))
    ref = delta.backward(rdx, *host(p, *INPUTS), scale=d ** -0.5)
    # fp32: errors add up over three kernels.  bf16: out and dx are rounded on
    # the way, so every gradient carries a few independent errors of h
    tol = 3e-5 if dtype == F32 else 6 * H8
    for g, r in zip((dgate, dw) + grads[:5], (rdgate, rdw) + tuple(ref[:5])):
        assert far(g, r)[0] <= tol


@pytest.mark.parametrize("dtype", [F32, BF])
def test_repeat_is_bitwise_and_nothing_is_written_outside(dtype):
    p = problem(2, 4, 2, 131, 64, 64, dtype, 19)
    args = [p[n] for n in INPUTS]
    need = la.la_delta_backward_workspace_size(2, 4, 2, 131, 64, 64, dtype)
    ws = torch.full((need + 512,), 0x5A, dtype=torch.uint8, device="cuda")
    first = la.la_backward_delta(p["dout"], *args, S0=p["S0"], dS_out=p["dS_out"], workspace=ws[:need])
    assert bool((ws[need:] == 0x5A).all())
    ws.random_(0, 256)  # what the scratch holds does not matter
    again = la.la_backward_delta(p["dout"], *args, S0=p["S0"], dS_out=p["dS_out"], workspace=ws[:need])
    for a, b in zip(first, again):
        assert torch.equal(a, b)
    need = la.la_delta_workspace_size(2, 4, 2, 131, 64, 64, dtype)
    band = torch.full((2 * 4 * 131 * 64 + 128,), 7.0, dtype=dtype, device="cuda")
    out = band[:-128].view(2, 4, 131, 64)
    ws = torch.full((need + 512,), 0x5A, dtype=torch.uint8, device="cuda")
    la.la_forward_delta(*args, out, S0=p["S0"], workspace=ws[:need] if need else None)
    assert bool((band[-128:] == 7.0).all()) and bool((ws[need:] == 0x5A).all())
    ws.random_(0, 256)
    o2, _ = la.la_forward_delta(*args, S0=p["S0"], workspace=ws[:need] if need else None)
    assert torch.equal(out, o2)


@pytest.mark.parametrize("dtype", [F32, BF])
def test_future_tokens_do_not_reach_back(dtype):
    p = problem(1, 2, 2, 150, 64, 64, dtype, 20)
    args = [p[n] for n in INPUTS]
    out, _ = la.la_forward_delta(*args, S0=p["S0"])
    for x in args:
        x[:, :, 100:] = -x[:, :, 100:].abs() if x is p["log_alpha"] else x[:, :, 100:] * 0.5
    o2, _ = la.la_forward_delta(*args, S0=p["S0"])
    assert torch.equal(out[:, :, :100], o2[:, :, :100])
    assert not torch.equal(out[:, :, 100:], o2[:, :, 100:])


def test_another_stream():
    """Arguments made on one stream, the call on another, its results used on
    the first after a wait; scratch comes from the call's own stream."""
    p = problem(2, 4, 4, 700, 128, 128, BF, 21)
    args = [p[n] for n in INPUTS]
    out, S = la.la_forward_delta(*args, S0=p["S0"], return_state=True)
    grads = la.la_backward_delta(p["dout"], *args, S0=p["S0"])
    side = torch.cuda.Stream()
    for handle in (side, side.cuda_stream):
        o, s = la.la_forward_delta(*args, S0=p["S0"], return_state=True, stream=handle)
        g = la.la_backward_delta(p["dout"], *args, S0=p["S0"], stream=handle)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(o, out) and torch.equal(s, S)
        assert all(torch.equal(a, b) for a, b in zip(g, grads) if a is not None)


def test_two_captured_graphs():
    """Two graphs with a workspace each, replayed in turn and at once on two
    streams, equal the eager calls."""
    runs = []
    for seed in (22, 23):
        p = problem(1, 4, 2, 300, 64, 64, BF, seed)
        args = [p[n] for n in INPUTS]
        eager, _ = la.la_forward_delta(*args, S0=p["S0"])
        grads = la.la_backward_delta(p["dout"], *args, S0=p["S0"])
        ws = torch.empty(max(16, la.la_delta_workspace_size(1, 4, 2, 300, 64, 64, BF)),
                         dtype=torch.uint8, device="cuda")
        wb = torch.empty(la.la_delta_backward_workspace_size(1, 4, 2, 300, 64, 64, BF),
                         dtype=torch.uint8, device="cuda")
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out, _ = la.la_forward_delta(*args, S0=p["S0"], workspace=ws)
            got = la.la_backward_delta(p["dout"], *args, S0=p["S0"], workspace=wb)
        runs.append((graph, out, got, eager, grads, p, ws, wb))
    side = torch.cuda.Stream()
    for _ in range(3):
        for r in runs:
            r[1].zero_()
            for g in r[2]:
                g.zero_()
        side.wait_stream(torch.cuda.current_stream())
        runs[0][0].replay()
        with torch.cuda.stream(side):
            runs[1][0].replay()
        torch.cuda.synchronize()
        for _, out, got, eager, grads, *_ in runs:
            assert torch.equal(out, eager)
            assert all(torch.equal(a, b) for a, b in zip(got, grads))


def test_captured_decode():
    p = problem(4, 4, 2, 6, 64, 64, BF, 24)
    S, Sg = p["S0"].clone(), p["S0"].clone()
    x = [p[n][:, :, 0].contiguous() for n in INPUTS]
    out = torch.empty(4, 4, 64, dtype=BF, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        la.la_decode_step_delta(Sg, *x, out)
    for t in range(6):
        now = [p[n][:, :, t].contiguous() for n in INPUTS]
        for a, b in zip(x, now):
            a.copy_(b)
        graph.replay()
        assert torch.equal(la.la_decode_step_delta(S, *now), out)
    assert torch.equal(S, Sg)


def test_refusals_of_the_binding():
    p = problem(1, 4, 2, 8, 64, 64, BF, 25)
    a = [p[n] for n in INPUTS]
    with pytest.raises(ValueError):
        la.la_forward_delta(a[0][:, :1].contiguous(), *a[1:])
    with pytest.raises(ValueError):
        la.la_forward_delta(a[0].transpose(2, 3), *a[1:])
    with pytest.raises(TypeError):
        la.la_forward_delta(a[0].float(), *a[1:])
    with pytest.raises(TypeError):
        la.la_forward_delta(a[0], a[1], a[2], a[3].double(), a[4])
    with pytest.raises(TypeError):
        la.la_forward_delta(a[0].half(), a[1].half(), a[2].half(), a[3])
    with pytest.raises(ValueError):
        la.la_forward_delta(*a, S0=p["S0"][:, :2].contiguous())
    with pytest.raises(ValueError):
        la.la_forward_delta(a[0], a[1], a[2], a[3].cpu())
    with pytest.raises(la.LinAttnError):
        la.la_forward_delta(*a, feature_map="elu1")
    with pytest.raises(la.LinAttnError):
        la.la_backward_delta(p["dout"], *a, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        la.la_backward_delta(p["dout"][:, :, :4].contiguous(), *a)
    with pytest.raises(ValueError):
        la.la_decode_step_delta(p["S0"], *a)
    with pytest.raises(ValueError):
        la.la_norm_gate(p["dout"], p["dout"])


def test_backward_with_a_loss_scale():
    """Output gradients of 2^16 and more beside rows that get none (beta = 0, no
    state yet): scales of operands that are zero multiply scales of large ones."""
    p = problem(1, 2, 2, 130, 64, 64, BF, 26, state=False)
    p["dout"] = (p["dout"].float() * 2.0 ** 18).to(BF)
    p["beta"][:, :, :3] = 0
    p["beta"][:, :, 64:70] = 0
    check_backward(p)
    p["dout"] = (p["dout"].float() * 2.0 ** -70).to(BF)
    check_backward(p)


@pytest.mark.parametrize("B,H,Hk,N,d,dv", [(10, 8, 4, 150, 64, 64), (40, 2, 1, 97, 128, 128),
                                           (160, 2, 2, 70, 32, 32), (13, 12, 12, 66, 64, 128)])
def test_many_heads(B, H, Hk, N, d, dv):
    """More 16-column slices than the GPU gives two warps each: one warp per
    slice, several slices per CTA."""
    p = problem(B, H, Hk, N, d, dv, BF, B + d)
    check_forward(p)
    check_backward(p)


@pytest.mark.parametrize("B,H,Hk,N,d,dv", [(3, 8, 2, 900, 64, 64), (2, 6, 6, 1100, 128, 32),
                                           (4, 12, 2, 333, 32, 128)])
def test_backward_more_chunks_than_sms(B, H, Hk, N, d, dv):
    """Each CTA of the dQ, dK kernel takes several chunks, and several value heads
    of each."""
    check_backward(problem(B, H, Hk, N, d, dv, BF, N + dv))


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("B,H,Hk,N,d,dv,gated,state", [
    (1, 1, 1, 2048, 64, 64, True, True), (1, 2, 1, 2100, 128, 32, True, False),
    (1, 3, 3, 2623, 32, 128, False, True), (2, 1, 1, 3000, 64, 128, True, True),
    (1, 4, 2, 2561, 128, 128, True, True), (1, 1, 1, 2111, 32, 32, True, False)])
def test_few_sequences_in_segments(B, H, Hk, N, d, dv, gated, state, dtype):
    """Few heads over many chunks: segments that run at once from the states their
    ends' maps give; the last segment is short."""
    p = problem(B, H, Hk, N, d, dv, dtype, N, gated, state)
    check_forward(p)
    check_backward(p)
    _, S = la.la_forward_delta(None, *(p[n] for n in INPUTS[1:]), S0=p["S0"])
    St = torch.zeros_like(S) if p["S0"] is None else p["S0"].clone()
    _, S2 = la.la_forward_delta(*(p[n] for n in INPUTS), S0=St, S_out=St)
    # the state-only run and the run with outputs differ in nothing that enters S
    assert torch.equal(S, S2)


def test_an_output_in_an_inputs_place_is_refused():
    x = torch.zeros(1, 2, 40, 64, device="cuda", dtype=BF)
    b = torch.zeros(1, 2, 40, device="cuda")
    for kw in (dict(q=x.clone(), k=x.clone(), v=x), dict(q=x, k=x.clone(), v=x.clone()),
               dict(q=x.clone(), k=x, v=x.clone())):
        with pytest.raises(ValueError, match="shares"):
            la.la_forward_delta(*kw.values(), b, out=x)
        with pytest.raises(ValueError, match="shares"):
            y = x[:, :, 0].contiguous()
            one = {n: y if t is x else t[:, :, 0].contiguous() for n, t in kw.items()}
            la.la_decode_step_delta(torch.zeros(1, 2, 64, 64, device="cuda"), *one.values(),
                                    b[:, :, 0].contiguous(), out=y)


@pytest.mark.parametrize("dtype,H,N", [(BF, 2100, 8100), (F32, 16600, 1025)])
def test_offsets_past_32_bits(dtype, H, N):
    """v, out and their gradients hold more than 2^31 elements.  Every head has
    the same inputs and the same arithmetic, so every head's result is the
    first's bit for bit, and the first is right by a call of a few heads."""
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < (140 << 30):
        pytest.skip("needs 140 GB of device memory")
    g = torch.Generator(device="cuda").manual_seed(11)
    n = lambda *s: torch.randn(s, generator=g, device="cuda")
    q, k, v1, do1 = (n(1, 1, N, w).to(dtype) for w in (32, 32, 128, 128))
    beta1, la1 = torch.sigmoid(n(1, 1, N)), -torch.nn.functional.softplus(n(1, 1, N) - 2)
    few = 512  # enough heads for the same path: no segments, one warp per slice

    def run(heads):
        v, do, beta, gate = (t.expand(-1, heads, *t.shape[2:]).contiguous()
                             for t in (v1, do1, beta1, la1))
        out, S = la.la_forward_delta(q, k, v, beta, gate, return_state=True)
        return out, S, *la.la_backward_delta(do, q, k, v, beta, gate)[:5]

    want = run(few)
    got = run(H)
    assert got[0].numel() > 2 ** 31
    for i, (w, x) in enumerate(zip(want, got)):
        if i in (2, 3):  # dq, dk: sums over the heads that share the key head
            # fp32 sums of H equal numbers, one rounding to dtype on each side
            tol = torch.finfo(dtype).eps + 2 * H * 2.0 ** -24
            a, b = w.double() / few, x.double() / H
            assert (a - b).norm() <= tol * a.norm(), i
            continue
        assert torch.equal(x[:, :1], w[:, :1]), i
        for h in range(1, H, 64):
            part = x[:, h:h + 64]
            assert torch.equal(part, x[:, :1].expand_as(part)), (i, h)


def test_decode_offsets_past_32_bits():
    """The states hold more than 2^31 elements."""
    B, H = 131073 // 3, 3
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < (30 << 30):
        pytest.skip("needs 30 GB of device memory")
    g = torch.Generator(device="cuda").manual_seed(12)
    n = lambda *s: torch.randn(s, generator=g, device="cuda")
    S1, q1, k1, v1 = n(1, H, 128, 128), n(1, H, 128).to(BF), n(1, H, 128).to(BF), n(1, H, 128).to(BF)
    b1, a1 = torch.sigmoid(n(1, H)), -torch.sigmoid(n(1, H))
    many = lambda t: t.expand(B, *t.shape[1:]).contiguous()
    S = many(S1)
    assert S.numel() > 2 ** 31
    out = la.la_decode_step_delta(S, *(many(t) for t in (q1, k1, v1, b1, a1)))
    want = la.la_decode_step_delta(S1, q1, k1, v1, b1, a1)
    assert torch.equal(out, want.expand_as(out))
    for i in range(0, B, 4096):
        part = S[i:i + 4096]
        assert torch.equal(part, S1.expand_as(part)), i


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("N", [1, 2, 130])
def test_the_first_gate_of_a_zero_start_has_no_gradient(N, dtype):
    """It multiplies a zero state: exactly 0, which is all there is at N = 1."""
    p = problem(2, 4, 2, N, 64, 64, dtype, 14, state=False)
    got = check_backward(p)
    assert (got[4][:, :, 0] == 0).all()
    if N > 1:
        assert (got[4][:, :, 1:] != 0).any()


@pytest.mark.parametrize("N", [3, 7, 13, 40, 63])
@pytest.mark.parametrize("d,dv", [(128, 64), (32, 128)])
def test_short_sequences_of_many_heads(N, d, dv):
    """Both sides of the lengths where the forward changes its kernels."""
    p = problem(24, 16, 4, N, d, dv, BF, N + d)
    check_forward(p)
    check_backward(p)


@pytest.mark.parametrize("d", [64, 128])
def test_many_heads_of_32_columns(d):
    """Two warps per slice although there are more slices than SMs."""
    p = problem(20, 16, 8, 140, d, 32, BF, d)
    check_forward(p)
    check_backward(p)


@pytest.mark.parametrize("B,H,Hk,N,d,dv", [(10, 16, 4, 100, 128, 128), (13, 12, 6, 190, 64, 128),
                                           (80, 4, 1, 77, 128, 64)])
def test_a_few_heads_more_than_a_round(B, H, Hk, N, d, dv):
    """The heads of the last round of CTAs run two warps per slice, in a launch
    of their own."""
    p = problem(B, H, Hk, N, d, dv, BF, B)
    check_forward(p)
    check_backward(p)
