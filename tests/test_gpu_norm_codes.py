"""The norm's 8-bit codes against exact quotients.

v / s is 448 h w / max|h w| of its group: the row's factor cancels.  In fp32 h, h w, the maximum, its reciprocal's
product and the quotient are rounded, six roundings of 2^-24 with the two of h, below 2^-21 together.  So a code is
the nearest one (ties to even) of some value within 2^-21 of the exact quotient: it differs from the quotient's own
only next to halfway, where h w of few bits often lie exactly."""

import numpy as np
import pytest
import torch

from oracle import few_bits_oracle as F
from oracle import mla_oracle as O
from test_gpu_few_bits import f64, norm_inputs, ok

pytestmark = pytest.mark.gpu

OFF = 2.0 ** -21


def e4m3(q):
    """The nearest E4M3 value, ties to even, of |q| <= 448 (1 + OFF)."""
    step = np.exp2(np.maximum(np.floor(np.log2(np.maximum(np.abs(q), 2.0 ** -30))), -6.0) - 3)
    return np.clip(np.rint(q / step) * step, -448, 448)


@pytest.mark.parametrize("T,D", [(32, 1536), (1500, 512), (700, 1544), (5, 7168), (300, 7168), (40, 16384)])
@pytest.mark.parametrize("residual", [False, True])
def test_codes_are_nearest_of_the_exact_quotient(T, D, residual):
    from mla_absorbed_decode_absorb_gb300 import ops
    x, r, w = norm_inputs(T, D, 3 * T + D, residual=residual)
    y8, s = ops.mla_rms_norm_fp8(x, w, 1e-6, r, None if r is None else torch.empty_like(r))
    h = f64(x) + (f64(r) if residual else 0.0)
    v = h * f64(w)
    q = 448.0 * v / F.per_column(F.group_max(v), D)
    got = O.e4m3_decode(y8.cpu().numpy())
    low, high = np.minimum(e4m3(q * (1 - OFF)), e4m3(q * (1 + OFF))), np.maximum(e4m3(q * (1 - OFF)), e4m3(q * (1 + OFF)))
    assert ((got >= low) & (got <= high)).all()
    # few quotients are that near halfway: the test is a strict one for all others
    assert (low != high).mean() < 2e-3
    again, s2 = ops.mla_rms_norm_fp8(x, w, 1e-6, r, None if r is None else torch.empty_like(r))
    assert torch.equal(again, y8) and torch.equal(s2, s)
    ok()
