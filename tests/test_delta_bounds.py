"""The bounds of bf16 results tell an operand of one fp16 part from one rounded to
bf16 (no GPU)."""
import numpy as np
import pytest

from delta_bounds import bf16, excess, within
from oracle import delta


def problem():
    r = np.random.default_rng(3)
    n = lambda *s: r.standard_normal(s)  # noqa: E731
    B, H, Hk, N, d, dv = 1, 2, 2, 150, 64, 64
    p = dict(q=n(B, Hk, N, d), k=n(B, Hk, N, d), v=n(B, H, N, dv), beta=r.uniform(0.1, 0.9, (B, H, N)),
             log_alpha=-np.log1p(np.exp(2 * n(B, H, N) - 2)), S0=0.3 * n(B, H, d, dv), scale=d ** -0.5)
    return p, n(B, H, N, dv), 0.3 * n(B, H, d, dv)


def test_bf16_of_the_oracle():
    x = np.random.default_rng(1).standard_normal(1000) * 10.0 ** np.arange(-5, 5).repeat(100)
    np.testing.assert_array_equal(delta._bf16(x), bf16(x))


def test_rounding_alone_and_fp16_parts_pass():
    p, _, _ = problem()
    ref, _ = delta.forward(**p)
    assert within("dv", bf16(ref), ref)
    noise = np.random.default_rng(2).uniform(-1, 1, ref.shape) * 2.0 ** -12
    assert within("out", bf16(ref * (1 + noise)), ref)


@pytest.mark.parametrize("plant", ["bf16_read", "bf16_state"])
def test_a_state_of_bf16_fails(plant):
    p, dout, dS = problem()
    ref, _ = delta.forward(**p)
    out, _ = delta.forward(**p, plant=plant)
    assert not within("out", bf16(out), ref), excess(bf16(out), ref)
    want = delta.backward(dout, **p, dS_out=dS)
    got = delta.backward(dout, **p, dS_out=dS, plant=plant)
    assert not within("dq", bf16(got[0]), want[0]), excess(bf16(got[0]), want[0])


def test_written_values_of_bf16_fail():
    p, dout, dS = problem()
    want, got = (delta.backward(dout, **p, dS_out=dS, plant=x) for x in (None, "bf16_written"))
    assert not within("dk", bf16(got[1]), want[1]), excess(bf16(got[1]), want[1])


def test_a_missing_term_of_half_a_percent_fails():
    p, _, _ = problem()
    ref, _ = delta.forward(**p)
    assert not within("out", bf16(ref * 0.995), ref) and not within("dq", bf16(ref * 0.995), ref)
