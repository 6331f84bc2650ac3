"""The oracle of the convolution and the selective scan against what the definitions
fix (no GPU): worked numbers, closed forms, differences for every gradient, and planted
mistakes."""
import numpy as np
import pytest

from oracle import ssm


def problem(seed=0, B=2, N=6, C=4, n=3, G=2):
    r = np.random.default_rng(seed)
    m = lambda *s: r.standard_normal(s)  # noqa: E731
    p = dict(x=m(B, N, C), delta=m(B, N, C) - 1, A=-r.uniform(0.2, 2, (C, n)), Bm=m(B, N, G, n), Cm=m(B, N, G, n),
             D=m(C), z=m(B, N, C), delta_bias=0.3 * m(C), S0=m(B, C, n))
    return p, m(B, N, C), m(B, C, n)


def check_two_tokens(plant=None):
    """One channel, one state, dt = 1 and 2 as given, A = -ln 2: S = 3 . 1 . 2 = 6, then
    6 / 4 + 2 . 5 . 1 = 11.5; out = C S + D x."""
    out, S = ssm.scan(np.array([[[3.0], [5.0]]]), np.array([[[1.0], [2.0]]]), np.array([[-np.log(2.0)]]),
                      np.array([2.0, 1.0]).reshape(1, 2, 1, 1), np.array([1.0, 2.0]).reshape(1, 2, 1, 1),
                      D=[10.0], softplus_on=False, plant=plant)
    np.testing.assert_allclose(out.ravel(), [36.0, 73.0], rtol=1e-14)
    np.testing.assert_allclose(S.ravel(), [11.5], rtol=1e-14)


def check_closed_form(plant=None):
    """S_t = exp(A sum_{1..t} dt) S_0 + sum_j exp(A sum_{j+1..t} dt) dt_j x_j B_j."""
    p, _, _ = problem(1)
    p.pop("z")
    out, S = ssm.scan(**p, plant=plant)
    dt = np.log1p(np.exp(p["delta"] + p["delta_bias"]))
    T = np.cumsum(dt, 1)
    B, N, C = p["x"].shape
    for c in range(C):
        g = c // 2
        for t in range(N):
            h = np.exp(p["A"][c] * T[:, t, c, None]) * p["S0"][:, c]
            for j in range(t + 1):
                h = h + (np.exp(p["A"][c] * (T[:, t, c] - T[:, j, c])[:, None])
                         * (dt[:, j, c] * p["x"][:, j, c])[:, None] * p["Bm"][:, j, g])
            y = (h * p["Cm"][:, t, g]).sum(-1) + p["D"][c] * p["x"][:, t, c]
            np.testing.assert_allclose(out[:, t, c], y, rtol=1e-11, atol=1e-12)
        np.testing.assert_allclose(S[:, c], h, rtol=1e-11, atol=1e-12)


def check_differences(plant=None):
    """Central differences of <out, dout> + <S, dS> (step 1e-5, error O(step^2)), with one
    row that ends early."""
    p, dout, dS = problem(2)
    lengths = [6, 4]

    def loss(q):
        out, S = ssm.scan(**q, lengths=lengths)
        return (out * dout).sum() + (S * dS).sum()

    g = ssm.scan(**p, lengths=lengths, dout=dout, dS_out=dS, plant=plant)
    for name, x in p.items():
        for i in np.random.default_rng(3).choice(x.size, min(x.size, 16), replace=False):
            at = np.unravel_index(i, x.shape)
            step = []
            for sign in (1e-5, -1e-5):
                y = x.copy()
                y[at] += sign
                step.append(loss(dict(p, **{name: y})))
            np.testing.assert_allclose(g[name][at], (step[0] - step[1]) / 2e-5, rtol=1e-6, atol=1e-7, err_msg=name)


def check_split(plant=None):
    """A sequence in two pieces, and a row that ends early, have the states of the tokens they hold."""
    p, _, _ = problem(4)
    out, S = ssm.scan(**p, plant=plant)
    first = {k: v[:, :4] if k in ("x", "delta", "Bm", "Cm", "z") else v for k, v in p.items()}
    rest = {k: v[:, 4:] if k in ("x", "delta", "Bm", "Cm", "z") else v for k, v in p.items()}
    o1, S1 = ssm.scan(**first, plant=plant)
    o2, S2 = ssm.scan(**dict(rest, S0=S1), plant=plant)
    np.testing.assert_allclose(np.concatenate([o1, o2], 1), out, rtol=1e-12)
    np.testing.assert_allclose(S2, S, rtol=1e-12)
    short, Ss = ssm.scan(**p, lengths=[4, 4], plant=plant)
    np.testing.assert_allclose(Ss, S1, rtol=1e-12)
    assert not short[:, 4:].any()


def check_conv_numbers(plant=None):
    """Three taps (1, 10, 100) over 1, 2, 3 with 5, 7 before: oldest first, the token last."""
    y, S = ssm.conv(np.array([[[1.0], [2.0], [3.0]]]), [[1.0, 10.0, 100.0]], [0.5], activation="none",
                    S0=[[[5.0], [7.0]]], plant=plant)
    np.testing.assert_allclose(y.ravel(), [175.5, 217.5, 321.5], rtol=1e-14)
    np.testing.assert_allclose(S.ravel(), [2.0, 3.0], rtol=0)


def check_conv_differences(plant=None):
    r = np.random.default_rng(5)
    p = dict(x=r.standard_normal((2, 5, 3)), weight=r.standard_normal((3, 4)), bias=r.standard_normal(3),
             S0=r.standard_normal((2, 3, 3)))
    dy, dS = r.standard_normal((2, 5, 3)), r.standard_normal((2, 3, 3))
    lengths = [5, 2]

    def loss(q):
        y, S = ssm.conv(**q, lengths=lengths, plant=plant)
        return (y * dy).sum() + (S * dS).sum()

    got = dict(zip(("x", "weight", "bias", "S0"), ssm.conv(**p, lengths=lengths, dy=dy, dS_out=dS, plant=plant)[2:]))
    for name, x in p.items():
        for at in np.ndindex(x.shape):
            step = []
            for sign in (1e-5, -1e-5):
                y = x.copy()
                y[at] += sign
                step.append(loss(dict(p, **{name: y})))
            np.testing.assert_allclose(got[name][at], (step[0] - step[1]) / 2e-5, rtol=1e-6, atol=1e-7, err_msg=name)


def check_conv_window(plant=None):
    """The window of a short row holds the row's own last inputs, older ones moved up."""
    x = np.arange(1.0, 6.0).reshape(1, 5, 1)
    _, S = ssm.conv(x, np.ones((1, 4)), S0=[[[-3.0], [-2.0], [-1.0]]], lengths=[1], plant=plant)
    np.testing.assert_allclose(S.ravel(), [-2.0, -1.0, 1.0])


CHECKS = [check_two_tokens, check_closed_form, check_differences, check_split, check_conv_numbers,
          check_conv_differences, check_conv_window]
PLANTS = ["undecayed", "input_not_stepped", "read_before_write", "decay_of_the_new_state",
          "softplus_not_differentiated", "taps_reversed", "window_ignores_length", "no_slope"]


@pytest.mark.parametrize("check", CHECKS)
def test_pin(check):
    check()


@pytest.mark.parametrize("plant", PLANTS)
def test_planted_mistake_is_caught(plant):
    failed = []
    for check in CHECKS:
        try:
            check(plant)
        except AssertionError:
            failed.append(check.__name__)
    assert failed, plant


def test_slopes():
    u = np.array([-700.0, -30.0, -1.0, 0.0, 1.0, 30.0, 700.0])
    for name in ("silu", "sigmoid", "none"):
        v, s = ssm.act(u, name)
        lo, hi = ssm.act(u - 1e-6, name)[0], ssm.act(u + 1e-6, name)[0]
        np.testing.assert_allclose(s, (hi - lo) / 2e-6, rtol=1e-6, atol=1e-7)
        assert np.all(np.isfinite(v))
