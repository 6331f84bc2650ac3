"""How far a bf16 result of the delta rule may be off (imported only by tests).

A result is rounded once to bf16.  What that alone costs is computed from the
reference: rho = |bf16(ref) - ref| / |ref|, about 1.66e-3 for normal values (a
rounding is off by at most 2^-8 of the value).  Errors before that rounding, far
under a step, add up with it as independent errors do: |got - ref|^2 = (rho^2 +
delta^2) |ref|^2.  delta counts fp16 operands of one part, each off by at most 2^-12
of a term, 2^-12 / sqrt(3) in the mean:
 - out: P, E and S, three of them: 2^-12; twice that for errors that are not
   independent: 2 parts.
 - dq, dk: three in each of the sums (E, dV, dS or S; the 64 x 64 matrix on its
   way; dO or a row image are exact), twice as above, and twice for sums whose
   terms cancel to half: 4 parts.
 - dv: fp32 until its rounding, the library's 1e-5 of the norm: 0.1 parts (2.4e-5).
An operand rounded to bf16 costs 16 parts / sqrt(3) of the terms it enters."""
import numpy as np
import torch

PARTS = {"out": 2.0, "dq": 4.0, "dk": 4.0, "dv": 0.1}


def bf16(x):
    return torch.from_numpy(np.ascontiguousarray(x)).to(torch.bfloat16).double().numpy()


def excess(got, ref):
    """delta in parts of 2^-12 (0 where the error is under the rounding's own)."""
    size = np.linalg.norm(ref)
    err, rho = np.linalg.norm(got - ref) / size, np.linalg.norm(bf16(ref) - ref) / size
    return float(np.sqrt(max(err ** 2 - rho ** 2, 0.0)) * 2.0 ** 12)


def within(name, got, ref):
    return bool(np.all(np.isfinite(got))) and excess(got, ref) <= PARTS[name]
