"""4-bit weights whose scales lie at and below 2^-100, down to bf16's smallest value: the quantiser rescales both sides
there, and codes are clamped where the scale itself is rounded coarsely.  Codes and scales are those of the
definition, bit for bit."""

import numpy as np
import pytest
import torch

from oracle import few_bits_oracle as F
from test_gpu_few_bits import f64, ok

pytestmark = pytest.mark.gpu

K = 128


def check(w):
    """w [N, K] float64 of bf16 values -> (u, scale) after the comparison."""
    from mla_absorbed_decode_absorb_gb300 import ops
    t = torch.tensor(w, dtype=torch.float32).to(torch.bfloat16)
    assert np.array_equal(f64(t), w)
    u, s = F.quantize_w4(w)
    w4, scale = ops.mla_quantize_w4(t.cuda())
    assert np.array_equal(f64(scale), s)
    assert np.array_equal(F.unpack_w4(w4.cpu().numpy()), u)
    back = ops.mla_dequantize_w4(w4, scale)
    assert np.array_equal(f64(back), F.bf16_round((u - 8) * F.per_column(s, w.shape[1])))
    ok()
    return u, s


@pytest.mark.parametrize("ragged", [0, 64])
def test_scales_of_few_bits(ragged):
    """Every scale b 2^-133, b = 1 .. 127, with the smallest and the largest maximum that has it and every weight up to
    that: ties, and quotients up to 10, which the clamp takes to -8 and 7."""
    rng = np.random.default_rng(1)
    rows = []
    for b in range(1, 128):
        m = np.arange(1, 2 ** 10)
        m = m[(np.rint(m / 7.0) == b) & (F.bf16_round(m * 2.0 ** -133) == m * 2.0 ** -133)]
        for top in (m.min(), m.max()):
            every = np.arange(top + 1)
            every = every[F.bf16_round(every * 2.0 ** -133) == every * 2.0 ** -133]
            for part in np.array_split(every, -(-len(every) // (K - 2))):
                row = np.concatenate([[top, -top], part, rng.choice(every, K - 2 - len(part))])
                rows.append(row * rng.choice([-1, 1], K))
    w = np.array(rows, np.float64) * 2.0 ** -133
    if ragged:
        w = np.concatenate([w, w[:, :ragged]], 1)
    u, s = check(w)
    q = w / F.per_column(s, w.shape[1])
    assert (u == 0).any() and (u == 15).any() and q.max() == 10 and q.min() == -10  # the clamp is reached
    assert (np.abs(q - np.rint(q)) == 0.5).any()
    assert (s < 2.0 ** -126).all()


def test_scales_on_both_sides_of_the_border():
    """Maxima of 2^-132 to 2^-96, scales on both sides of 2^-126 (bf16's normal range) and of 2^-100."""
    rng = np.random.default_rng(2)
    rows = []
    for e in range(-132, -95):
        for _ in range(8):
            row = rng.integers(128, 256, K) * 2.0 ** (e - 7 - rng.integers(0, 6, K)) * rng.choice([-1, 1], K)
            row[rng.integers(K)] = rng.integers(128, 256) * 2.0 ** (e - 7)
            rows.append(F.bf16_round(row))
        # the largest weight 7 s exactly and weights k s + s / 2: ties of either parity
        s = rng.integers(16, 32) * 2.0 ** (e - 7)
        rows.append(F.bf16_round(np.concatenate([[7 * s], (np.arange(K - 1) % 15 - 7.5) * s])))
    w = np.array(rows)
    w[np.abs(w) < 2.0 ** -133] = 0
    _, s = check(w)
    assert (s < 2.0 ** -126).any() and ((s >= 2.0 ** -126) & (s < 2.0 ** -100)).any() and (s >= 2.0 ** -100).any()
    border = F.bf16_round(np.array([127, 128, 129, 255, 256]) * 7 * 2.0 ** -107)
    _, s = check(np.concatenate([border[:, None], np.resize(border, (5, K - 1)) / 4], 1))
    assert (s == 2.0 ** -100).any() and (s < 2.0 ** -100).any() and (s > 2.0 ** -100).any()
