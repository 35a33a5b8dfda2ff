"""The 4-bit projections over long rows, with sums that fp32 holds exactly: nothing is allowed but y's rounding.

x is 0 or +-1, the weights are whole and the scales powers of two of one size, so every product and every partial sum
is a whole number below 2^24 in whatever order it is formed, and y is the rounded sum, bit for bit."""

import numpy as np
import pytest
import torch

from oracle import few_bits_oracle as F
from test_gpu_few_bits import f64, ok, run_linear

pytestmark = pytest.mark.gpu


def whole_inputs(T, K, N, fp8, seed):
    rng = np.random.default_rng(seed)
    x = rng.integers(-1, 2, (T, K)).astype(np.int8)
    if K > 2 ** 21:
        x[:, rng.integers(0, 4, K) > 0] = 0  # a quarter of the columns: |sum| <= 8 K / 4
    u = rng.integers(0, 16, (N, K)).astype(np.uint8)
    assert 8 * np.abs(x.astype(np.int64)).sum(1).max() < 2 ** 24
    w4 = torch.tensor(F.pack_w4(u))
    scale = torch.full((N, F.groups(K)), 0.25, dtype=torch.bfloat16)
    ref = np.zeros((T, N))
    half = np.zeros((T, N))
    for k in range(0, K, 2 ** 18):
        ref += x[:, k:k + 2 ** 18].astype(np.float64) @ (u[:, k:k + 2 ** 18].astype(np.float64) - 8).T
        if k < K // 2:
            stop = min(k + 2 ** 18, K // 2)
            half += x[:, k:stop].astype(np.float64) @ (u[:, k:stop].astype(np.float64) - 8).T
    ref, half = F.bf16_round(ref / 4), F.bf16_round(half / 4)
    # the comparison rejects zeros, a sum over half of K and a sum that lacks its last group
    assert (ref != 0).mean() > 0.9 and (ref != half).mean() > 0.9
    if fp8:
        codes = np.where(x == 0, 0, np.where(x > 0, 0x38, 0xb8)).astype(np.uint8)  # +-1
        return torch.tensor(codes), torch.ones(T, F.groups(K)), w4, scale, ref
    return torch.tensor(x).to(torch.bfloat16), None, w4, scale, ref


# Thousands of groups, few features: the warp kernel whole and divided, then the tensor-core kernel (over 36 M weights
# times passes of 8 tokens) at each of its tiles, up to the longest row that is taken.
@pytest.mark.parametrize("T,K,N", [
    (1, 262144, 3), (5, 65600, 40), (8, 16384, 130), (70, 262144, 3), (1, 4194304, 2), (3, 4194240, 1),
    (16, 262144, 70), (48, 262144, 23), (64, 262144, 18), (100, 262144, 11), (256, 16384, 130), (256, 262144, 5),
    (9, 4194304, 5), (70, 4194240, 1), (130, 1048640, 3)])
@pytest.mark.parametrize("fp8", [False, True])
def test_long_rows_are_summed_exactly(T, K, N, fp8):
    x, sx, w4, scale, ref = whole_inputs(T, K, N, fp8, T + N)
    y = run_linear(x, sx, w4, scale)
    assert np.array_equal(f64(y), ref)
    ok()
