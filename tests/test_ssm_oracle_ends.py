"""The scan's oracle behind a row's end (no GPU): nothing there is read, and what the last token
left is not either."""
import numpy as np
import pytest

from oracle import ssm

ROWS = ("x", "delta", "Bm", "Cm", "z")


def problem(lengths, N=7, C=4, n=3, G=2):
    r = np.random.default_rng(5)
    B = len(lengths)
    m = lambda *s: r.standard_normal(s)  # noqa: E731
    p = dict(x=m(B, N, C), delta=m(B, N, C) - 1, A=-r.uniform(0.2, 2, (C, n)), Bm=m(B, N, G, n), Cm=m(B, N, G, n),
             D=m(C), z=m(B, N, C), delta_bias=0.3 * m(C), S0=m(B, C, n))
    return p, m(B, N, C), m(B, C, n)


def test_nothing_behind_a_row_is_read():
    lengths = [0, 1, 4, 7]
    p, dout, dS = problem(lengths)
    want = ssm.scan(**p, lengths=lengths, dout=dout, dS_out=dS)
    for b, n in enumerate(lengths):
        for k in ROWS:
            p[k][b, n:] = np.nan
        dout[b, n:] = np.nan
    got = ssm.scan(**p, lengths=lengths, dout=dout, dS_out=dS)
    for k, w in want.items():
        np.testing.assert_array_equal(got[k], w, err_msg=k)


@pytest.mark.parametrize("name", ["x", "Bm"])
def test_a_last_state_of_nan_stays_in_its_row(name):
    """The last token's own input reaches the outputs of that token and the state, no rate's
    gradient (states before each token) and nothing behind the row."""
    lengths = [3, 7]
    p, dout, dS = problem(lengths)
    want = ssm.scan(**p, lengths=lengths, dout=dout, dS_out=dS)
    p[name][0, 2] = np.nan
    got = ssm.scan(**p, lengths=lengths, dout=dout, dS_out=dS)
    assert np.isnan(got["S"][0]).all()
    np.testing.assert_allclose(got["A"], want["A"], rtol=1e-14)
    for k in (*ROWS, "out"):
        assert not got[k][0, 3:].any(), k
        np.testing.assert_allclose(got[k][1], want[k][1], rtol=1e-14)
