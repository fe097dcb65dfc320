"""The activations of the dense products deep in their lower tail, where they are small
but representable: errors relative to the value, not to one.

Bounds, in units of 2^-23 relative to the value (or, for a slope, to the sum of its
terms' magnitudes), from the error bounds that CUDA gives for its functions:
  exp(-y)     2 + 1.2 y, and y / 2 for each rounding of y itself
  1 / v       2
  products    1/2 each, and 4 for the polynomial of the normal distribution's tail
GELU (y = z^2 / 2, one rounding; two reciprocal errors through the polynomial): 16 + z^2.
SiLU (y = |z|): 4 + 1.3 |z|.  tanh form (y = 2 sqrt(2 / pi) |z + 0.044715 z^3|, four
roundings): 4 + 3.3 y.  A slope has up to six more products: 6 more.
"""
import math

import pytest

from tests.test_gpu_dense_tokens import TYPES, act64, code, dt, rounding, within

pytestmark = pytest.mark.gpu

# from where the share p is a normal float32 number
LOWEST = {"gelu": -12.9, "gelu_tanh": -9.9, "silu": -86.0}


def tail_error(act, z):
    """Relative error of the share p that passes, in units of 2^-23."""
    if act == "gelu":
        return 16 + z * z
    if act == "silu":
        return 4 + 1.3 * z.abs()
    return 4 + 3.3 * 2 * math.sqrt(2 / math.pi) * (z.abs() + 0.044715 * z.abs() ** 3)


def exact(act, z):
    """(act(z), its slope's terms' magnitudes, act'(z)) in float64, without cancellation."""
    import torch
    if act == "silu":
        p = torch.special.expit(z)
        return z * p, p * (1 + z.abs() * (1 - p)), p * (1 + z * (1 - p))
    if act == "gelu":
        p = 0.5 * torch.special.erfc(-z / math.sqrt(2.0))
        d = z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
        return z * p, p + d.abs(), p + d
    c = 2 * math.sqrt(2 / math.pi)
    p = torch.special.expit(c * (z + 0.044715 * z ** 3))
    d = z * p * (1 - p) * c * (1 + 3 * 0.044715 * z * z)
    return z * p, p + d.abs(), p + d


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("act", ["gelu", "gelu_tanh", "silu"])
def test_lower_tails(sig, act, dtype):
    """An identity weight, so that the kernel's sum is the argument itself; 7 tokens for
    the few-token kernel's epilogue and 4300 for the pair kernel's."""
    import torch
    n = 512
    z = torch.linspace(LOWEST[act], 0.0, 4300 * n, dtype=torch.float64, device="cuda").to(dt(dtype)).reshape(n, 4300)
    z = z.T.contiguous()                                       # every row runs through the range
    z64 = z.double()
    keep = z64 >= LOWEST[act]
    eye, zero = torch.eye(n, dtype=dt(dtype), device="cuda"), torch.zeros(n, n, dtype=dt(dtype), device="cuda")
    a, mags, slope = exact(act, z64)
    assert bool(((a - act64(act, z64)[0]).abs() <= 1e-14).all())   # the same function, up to its cancellation
    rel = tail_error(act, z64) * 2.0 ** -23
    tol = rounding(a, rel * a.abs(), dtype)
    for rows in (7, 4300):
        got = sig.linear_act(z[:rows], eye, act=code(sig, act))
        within(torch.where(keep[:rows], got.double(), a[:rows]), a[:rows], tol[:rows], f"{act} of {rows}")
        # dX with dh = 1 (WdT = I, dY = 1), u = 1 and unit gate weights is act'(z)
        one = torch.ones_like(z[:rows])
        dX = sig.gated_mlp_backward(one, z[:rows], z[:rows], one, eye, zero, eye, act=code(sig, act),
                                    want_weights=False)[0]
        e = rounding(slope, (rel + 6 * 2.0 ** -23) * mags, dtype)
        within(torch.where(keep[:rows], dX.double(), slope[:rows]), slope[:rows], e[:rows], f"slope of {rows}")
