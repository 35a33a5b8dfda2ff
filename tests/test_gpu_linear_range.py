"""The 4-bit projections at the ends of the scales' range: what every group's sum and its scaled value fit, y has."""

import numpy as np
import pytest
import torch

from oracle import few_bits_oracle as F
from test_gpu_few_bits import f64, linear_inputs, linear_ref, ok, run_linear, within

pytestmark = pytest.mark.gpu

# (exponent of the weights' scales, of x's): y of about 2^16 to 2^26, near 1, and small
ENDS = [(125, -105), (120, -100), (-120, 110), (-100, -20), (0, -100), (-126, 108)]


@pytest.mark.parametrize("T,K,N", [(1, 320, 70), (8, 1024, 40), (9, 1088, 16601), (40, 320, 24000), (64, 320, 14500),
                                   (100, 1088, 2600), (256, 4160, 3000)])
@pytest.mark.parametrize("we,xe", ENDS)
def test_scales_at_the_ends_of_their_range(T, K, N, we, xe):
    """8-bit x with scales of about 2^xe and weights with scales of about 2^we (the largest the quantiser writes, 2^125,
    and below bf16's normal range): a scale is not multiplied by anything that leaves fp32's range by itself.  The
    tolerance is that of the ordinary sizes, times the same power of two."""
    x, sx, w4, scale = linear_inputs(T, K, N, True, T + K)
    ref, tol = linear_ref(x, sx, w4, scale)
    up, down = np.ldexp(1.0, we), np.ldexp(1.0, xe)
    big = (scale.double() * up).to(torch.bfloat16)
    bx = (sx.double() * down).to(torch.float32)
    if we < -117:  # scales that lost bits below the normal range
        ref, tol = linear_ref(x, bx, w4, big)
    else:
        assert np.array_equal(f64(big), f64(scale) * up) and np.array_equal(bx.double().numpy(), sx.double().numpy() * down)
        ref, tol = ref * up * down, tol * up * down
    # Below 2^-126 a bf16 value is a multiple of 2^-133, so y is off by up to 2^-134 there whatever the sums.  The sums
    # of 8-bit x are kept times 2^-9: an fp32 rounding below 2^-126 is at most 2^-150, 2^-141 of y, and a group makes at
    # most three of them (product, addition, a cluster's addition).
    tol = tol + 2.0 ** -134 + 3 * F.groups(K) * 2.0 ** -141
    assert np.abs(ref).max() < 2.0 ** 120
    y = run_linear(x, bx, w4, big)
    within(f64(y), ref, tol)
    ok()
