"""The delta-rule oracle against what the definition fixes (no GPU): the
printed comparison of additive and corrected writes, the explicit solve of one
chunk, differences for every gradient, and planted mistakes."""
import numpy as np
import pytest

from oracle import delta


def problem(seed=0, B=2, H=4, Hk=2, N=7, d=5, dv=3):
    r = np.random.default_rng(seed)
    n = lambda *s: r.standard_normal(s)  # noqa: E731
    return dict(q=n(B, Hk, N, d), k=n(B, Hk, N, d), v=n(B, H, N, dv),
                beta=r.uniform(0.1, 1.0, (B, H, N)), log_alpha=-r.uniform(0, 0.7, (B, H, N)),
                S0=n(B, H, d, dv), scale=0.6), n(B, H, N, dv), n(B, H, d, dv)


def check_repeated_key(plant=None):
    """Writing 3, then 4 under one unit key with beta = 1: the additive state
    reads 7, the delta rule's reads 4, the last value."""
    k = np.ones((1, 1, 2, 1))
    v = np.array([3.0, 4.0]).reshape(1, 1, 2, 1)
    out, S = delta.forward(k, k, v, np.ones((1, 1, 2)), scale=1.0, l2=False, plant=plant)
    np.testing.assert_allclose(out.ravel(), [3.0, 4.0], atol=1e-15)
    np.testing.assert_allclose(S.ravel(), [4.0], atol=1e-15)


def check_dense(plant=None):
    """All tokens at once: E = (I + A diag(beta))^{-1} (V - diag(e^G) K S0)."""
    p, _, _ = problem()
    out, S = delta.forward(p["q"], p["k"], p["v"], p["beta"], p["log_alpha"], scale=p["scale"],
                           S0=p["S0"], plant=plant)
    unit = lambda x: x / np.sqrt((x ** 2).sum(-1, keepdims=True) + 1e-6)  # noqa: E731
    N = p["v"].shape[2]
    for b in range(2):
        for h in range(4):
            q, k = unit(p["q"][b, h // 2]) * p["scale"], unit(p["k"][b, h // 2])
            G = np.cumsum(p["log_alpha"][b, h])
            D = np.tril(np.exp(np.minimum(G[:, None] - G[None, :], 0)))
            A = np.tril(D * (k @ k.T), -1)
            S0 = p["S0"][b, h]
            E = np.linalg.solve(np.eye(N) + A * p["beta"][b, h][None, :],
                                p["v"][b, h] - np.exp(G)[:, None] * (k @ S0))
            U = p["beta"][b, h][:, None] * E
            np.testing.assert_allclose(out[b, h], np.exp(G)[:, None] * (q @ S0) + (D * (q @ k.T)) @ U,
                                       atol=1e-12)
            np.testing.assert_allclose(S[b, h], np.exp(G[-1]) * S0
                                       + (np.exp(G[-1] - G)[:, None] * k).T @ U, atol=1e-12)


def check_differences(plant=None):
    """Every gradient against central differences of <out, dout> + <S, dS>
    (step 1e-5, error O(step^2) on values of order one)."""
    p, dout, dS = problem(1)

    def loss(p):
        out, S = delta.forward(p["q"], p["k"], p["v"], p["beta"], p["log_alpha"], scale=p["scale"],
                               S0=p["S0"])
        return (out * dout).sum() + (S * dS).sum()

    got = delta.backward(dout, p["q"], p["k"], p["v"], p["beta"], p["log_alpha"], scale=p["scale"],
                         S0=p["S0"], dS_out=dS, plant=plant)
    r = np.random.default_rng(5)
    for name, g in zip(("q", "k", "v", "beta", "log_alpha", "S0"), got):
        for _ in range(12):
            at = tuple(r.integers(0, n) for n in g.shape)
            two = []
            for step in (1e-5, -1e-5):
                x = dict(p)
                x[name] = p[name].copy()
                x[name][at] += step
                two.append(loss(x))
            assert abs((two[0] - two[1]) / 2e-5 - g[at]) < 1e-7, (name, at)


PINS = [check_repeated_key, check_dense, check_differences]


@pytest.mark.parametrize("pin", PINS, ids=lambda f: f.__name__)
def test_pin(pin):
    pin()


@pytest.mark.parametrize("plant", ["undecayed_error", "additive", "read_before_write",
                                   "key_only_written", "norm_not_differentiated"])
def test_planted_mistake_is_caught(plant):
    caught = 0
    for pin in PINS:
        try:
            pin(plant)
        except AssertionError:
            caught += 1
    assert caught


def test_state_splits_the_sequence():
    p, _, _ = problem(2)
    cut = lambda x, lo, hi: x[:, :, lo:hi]  # noqa: E731
    whole, S = delta.forward(*(p[n] for n in ("q", "k", "v", "beta", "log_alpha")),
                             scale=p["scale"], S0=p["S0"])
    a, Sa = delta.forward(*(cut(p[n], 0, 3) for n in ("q", "k", "v", "beta", "log_alpha")),
                          scale=p["scale"], S0=p["S0"])
    b, Sb = delta.forward(*(cut(p[n], 3, 7) for n in ("q", "k", "v", "beta", "log_alpha")),
                          scale=p["scale"], S0=Sa)
    np.testing.assert_allclose(np.concatenate([a, b], 2), whole, atol=1e-14)
    np.testing.assert_allclose(Sb, S, atol=1e-14)


@pytest.mark.parametrize("activation", ["silu", "sigmoid", "none"])
@pytest.mark.parametrize("per_head", [False, True])
def test_norm_gate_differences(activation, per_head):
    r = np.random.default_rng(3)
    x, gate, dy = r.standard_normal((2, 3, 4, 8)), r.standard_normal((2, 4, 3, 8)), \
        r.standard_normal((2, 4, 3, 8))
    w = r.standard_normal((3, 8) if per_head else 8)
    y, dx, dgate, dw = delta.norm_gate(x, gate, w, activation=activation, dy=dy)
    np.testing.assert_allclose(np.sqrt((delta.norm_gate(x) ** 2).mean(-1)), 1.0, atol=1e-4)
    p = {"x": x, "gate": gate, "weight": w}
    for name, g in (("x", dx), ("gate", dgate), ("weight", dw)):
        for _ in range(10):
            at = tuple(r.integers(0, n) for n in g.shape)
            two = []
            for step in (1e-5, -1e-5):
                z = dict(p)
                z[name] = p[name].copy()
                z[name][at] += step
                two.append((delta.norm_gate(z["x"], z["gate"], z["weight"],
                                            activation=activation) * dy).sum())
            assert abs((two[0] - two[1]) / 2e-5 - g[at]) < 1e-7, (name, at)
