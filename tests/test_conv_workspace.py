"""The workspace of the convolution's gradient holds a part for every block row of its launch,
down to one channel (no GPU)."""
import subprocess
import sys

import pytest

THREADS, PER_SM, SMS = 128, 4, 152  # of the gradient's launch


def parts(B, N, C, width):
    """Block rows of a launch with `width` channels a thread."""
    columns = -(-(C // width) // THREADS)
    rows = max(1, PER_SM * SMS // columns)
    run = max(8, -(-N // max(1, rows // B)))
    return min(rows, B * -(-N // run))


@pytest.fixture(scope="module")
def sizes():
    """(B, N, C, W) -> bytes, asked in a process of its own: an arithmetic fault ends that one."""
    from kernelised_causal_linear_gb300 import build

    build.build()
    cases = [(B, N, C, W) for B, N in ((1, 4096), (3, 5003), (700, 5), (1, 1))
             for C in (1, 2, 3, 4, 5, 6, 127, 128, 129, 511, 512, 513, 514, 2048) for W in (2, 4)]
    code = ("from kernelised_causal_linear_gb300._binding import raw\n"
            f"print([raw.la_conv_backward_workspace_size(*c, d) for c in {cases} for d in (0, 1)])")
    run = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert run.returncode == 0, (run.returncode, run.stderr)
    got = eval(run.stdout)  # noqa: S307  (a list of numbers)
    return {(*c, d): got[2 * i + d] for i, c in enumerate(cases) for d in (0, 1)}


def test_every_width_fits(sizes):
    for (B, N, C, W, dtype), got in sizes.items():
        need = max(parts(B, N, C, v) for v in (1, 2, 4) if C % v == 0) * (W + 1) * C * 4
        assert got >= need, (B, N, C, W, dtype, got, need)
