"""The norm with gate on the GPU against fp64.

Tolerances: every sum is fp32 over at most 128 terms of a row, and dweight over
the rows in a tree of fp32 sums: 1e-5 of the tensor's 2-norm and largest entry.
A bf16 result is rounded once, at most 2^-8 of the value per element."""
import numpy as np
import pytest
import torch

from gpu_util import to_np
from oracle import delta

pytestmark = pytest.mark.gpu

la = pytest.importorskip("kernelised_causal_linear_gb300")
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.fail("GPU test run without a CUDA device")
    yield
    assert la.la_get_device_status() == 0


def problem(B, H, N, dv, x_dtype, dtype, per_head, seed=0):
    g = torch.Generator().manual_seed(2000 + seed)
    n = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    return (n(B, H, N, dv).to(x_dtype).cuda(), (2 * n(B, N, H, dv)).to(dtype).cuda(),
            (1 + 0.2 * n(*((H, dv) if per_head else (dv,)))).cuda(), n(B, N, H, dv).to(dtype).cuda())


def assert_near(got, ref, what):
    g, r = to_np(got), np.asarray(ref)
    assert g.shape == r.shape and np.all(np.isfinite(g))
    if not g.size:
        return
    e = np.abs(g - r)
    slack = 1e-5 * np.abs(r).max()
    half = 2.0 ** -8 if got.dtype == BF else 0.0
    assert np.all(e <= half * np.abs(r) + slack), (what, e.max())
    if not half:
        assert np.linalg.norm(e) <= 1e-5 * np.linalg.norm(r), what


def check(x, gate, w, dy, activation, eps=1e-6):
    h = lambda t: None if t is None else to_np(t)  # noqa: E731
    y = la.la_norm_gate(x, gate, w, activation=activation, eps=eps,
                        y=None if gate is not None else torch.empty_like(dy))
    dx, dgate, dw = la.la_norm_gate_backward(dy, x, gate, w, activation=activation, eps=eps)
    ry, rdx, rdgate, rdw = delta.norm_gate(h(x), h(gate), h(w), activation=activation, eps=eps,
                                           dy=h(dy))
    assert_near(y, ry, "y")
    assert_near(dx, rdx, "dx")
    if gate is None:
        assert dgate is None
    else:
        assert_near(dgate, rdgate, "dgate")
    if w is None:
        assert dw is None
    else:
        assert_near(dw, rdw, "dweight")


@pytest.mark.parametrize("x_dtype", [F32, BF])
@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("dv", [32, 64, 128])
@pytest.mark.parametrize("B,H,N", [(1, 1, 1), (2, 3, 17), (3, 5, 130), (1, 2, 1000)])
def test_sizes(B, H, N, dv, dtype, x_dtype):
    check(*problem(B, H, N, dv, x_dtype, dtype, False, N + dv), "silu")


@pytest.mark.parametrize("activation", ["silu", "sigmoid", "none"])
@pytest.mark.parametrize("per_head", [False, True])
def test_options(activation, per_head):
    check(*problem(2, 4, 99, 64, F32, BF, per_head, 1), activation, eps=1e-2)


def test_without_gate_or_weight():
    x, gate, w, dy = problem(2, 3, 40, 128, BF, F32, False, 2)
    check(x, None, w, dy, "silu")
    check(x, gate, None, dy, "silu")
    check(x, None, None, dy, "silu")
    assert la.la_norm_gate(x).dtype == BF


def test_zero_rows_and_far_gates():
    """A zero row has y = 0 and a gradient of c / sqrt(eps); gates of +-1e4
    saturate without a NaN."""
    x, gate, w, dy = problem(1, 2, 20, 64, F32, F32, False, 3)
    gate[:, 3] = 1e4
    gate[:, 4] = -1e4
    check(x, gate, w, dy, "silu")
    check(x, gate, w, dy, "sigmoid")
    x[:, :, 5] = 0
    y = la.la_norm_gate(x, gate, w)
    assert not y[:, 5].any() and torch.isfinite(y).all()
    dx, _, _ = la.la_norm_gate_backward(dy, x, gate, w)
    _, rdx, _, _ = delta.norm_gate(to_np(x), to_np(gate), to_np(w), dy=to_np(dy))
    assert_near(dx[:, :, 5], rdx[:, :, 5], "dx")


def test_many_rows_repeat_bitwise():
    x, gate, w, dy = problem(3, 7, 5003, 32, BF, BF, True, 4)
    a = la.la_norm_gate_backward(dy, x, gate, w)
    need = la.la_norm_gate_backward_workspace_size(3, 7, 5003, 32)
    ws = torch.randint(0, 256, (need + 512,), dtype=torch.uint8, device="cuda")
    tail = ws[need:].clone()
    b = la.la_norm_gate_backward(dy, x, gate, w, workspace=ws[:need])
    assert all(torch.equal(p, q) for p, q in zip(a, b)) and torch.equal(ws[need:], tail)
    check(x, gate, w, dy, "silu")


@pytest.mark.parametrize("B,H,N,dv", [(1, 7, 3, 32), (2, 33, 29, 64), (1, 130, 11, 128),
                                      (3, 64, 40, 32), (1, 1, 5000, 128), (2, 48, 333, 64)])
def test_head_counts(B, H, N, dv):
    """Weights for each head with head counts that do and do not divide a block's
    rows, more heads than rows per block among them."""
    check(*problem(B, H, N, dv, F32, F32, True, H), "silu")
    check(*problem(B, H, N, dv, BF, BF, False, H), "sigmoid")


def test_no_tokens():
    x, gate, w, dy = problem(2, 3, 0, 64, F32, F32, True, 5)
    assert la.la_norm_gate(x, gate, w).shape == (2, 0, 3, 64)
    dx, dgate, dw = la.la_norm_gate_backward(dy, x, gate, w)
    assert dx.numel() == 0 and dgate.numel() == 0 and not dw.any()


def test_graph_and_stream():
    x, gate, w, dy = problem(2, 4, 300, 128, BF, BF, False, 6)
    y = la.la_norm_gate(x, gate, w)
    grads = la.la_norm_gate_backward(dy, x, gate, w)
    side = torch.cuda.Stream()
    y2 = la.la_norm_gate(x, gate, w, stream=side)
    g2 = la.la_norm_gate_backward(dy, x, gate, w, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(y, y2) and all(torch.equal(a, b) for a, b in zip(grads, g2))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y3 = la.la_norm_gate(x, gate, w)
        g3 = la.la_norm_gate_backward(dy, x, gate, w)
    for _ in range(2):
        y3.zero_()
        graph.replay()
        assert torch.equal(y, y3) and all(torch.equal(a, b) for a, b in zip(grads, g3))


def test_an_output_in_an_inputs_place_is_refused():
    x = torch.zeros(1, 2, 2, 64, device="cuda", dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="shares"):
        la.la_norm_gate(x, x.clone(), y=x)
    with pytest.raises(ValueError, match="shares"):
        la.la_norm_gate(x.clone(), x, y=x)


def test_offsets_past_32_bits():
    """More than 2^31 elements: every batch row has the same inputs, so the same
    results bit for bit, and the first row's are those of a call of its own."""
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < (60 << 30):
        pytest.skip("needs 60 GB of device memory")
    B, H, N, dv = 257, 8, 8192, 128
    g = torch.Generator(device="cuda").manual_seed(13)
    n = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()
    x1, g1, dy1 = n(1, H, N, dv), n(1, N, H, dv), n(1, N, H, dv)
    w = torch.randn(H, dv, generator=g, device="cuda")
    many = lambda t: t.expand(B, *t.shape[1:]).contiguous()
    x, gate, dy = many(x1), many(g1), many(dy1)
    assert x.numel() > 2 ** 31
    got = (la.la_norm_gate(x, gate, w), *la.la_norm_gate_backward(dy, x, gate, w)[:2])
    want = (la.la_norm_gate(x1, g1, w), *la.la_norm_gate_backward(dy1, x1, g1, w)[:2])
    for a, b in zip(got, want):
        for i in range(0, B, 32):
            part = a[i:i + 32]
            assert torch.equal(part, b.expand_as(part)), i
