"""Plain float64 definitions of the layer's few-bit operators (test infrastructure only).

The root-mean-square norm with its 8-bit output, the 4-bit weight format, the
projection with such weights, and the FP8 cache read back.  numpy only; shares
no code with the CUDA path.
"""

from __future__ import annotations

import numpy as np

from . import mla_oracle as O

GROUP = 128
NORM_FLOOR = 2.0 ** -100


def groups(n: int) -> int:
    return -(-n // GROUP)


def per_column(scale: np.ndarray, columns: int) -> np.ndarray:
    """[rows, groups] -> [rows, columns]: each column's scale."""
    return np.repeat(scale, GROUP, axis=1)[:, :columns]


def group_max(v: np.ndarray) -> np.ndarray:
    rows, columns = v.shape
    p = np.zeros((rows, groups(columns) * GROUP))
    p[:, :columns] = np.abs(v)
    return p.reshape(rows, -1, GROUP).max(-1)


def rms_norm(x, weight, eps, residual=None):
    """(h, v): h = x + residual and v = h / sqrt(mean(h^2) + eps) * weight."""
    h = np.asarray(x, np.float64)
    if residual is not None:
        h = h + residual
    return h, h / np.sqrt((h * h).mean(1, keepdims=True) + eps) * weight


def norm_scale(v):
    """The 8-bit output's scale of each group: max(max|v| / 448, 2^-100)."""
    return np.maximum(group_max(v) / 448.0, NORM_FLOOR)


def bf16_round(v: np.ndarray) -> np.ndarray:
    """The nearest bf16 value, ties to even, of finite values below bf16's overflow (below 2^-126 the step is 2^-133)."""
    v = np.asarray(v, np.float64)
    step = np.maximum(np.frexp(v)[1], -125) - 8
    return np.ldexp(np.rint(np.ldexp(v, -step)), step)


def quantize_w4(w):
    """(u [N, K] in 0..15, scale [N, groups]) of weights w."""
    s = bf16_round(group_max(w) / 7.0)
    s[s == 0] = 1.0
    return np.clip(np.rint(w / per_column(s, w.shape[1])), -8, 7).astype(np.int64) + 8, s


def pack_w4(u):
    """Half bytes to bytes: column 2i low, column 2i + 1 high."""
    return (u[:, 0::2] | (u[:, 1::2] << 4)).astype(np.uint8)


def unpack_w4(w4):
    u = np.empty((w4.shape[0], 2 * w4.shape[1]), np.int64)
    u[:, 0::2], u[:, 1::2] = w4 & 15, w4 >> 4
    return u


def weights_w4(w4, scale):
    u = unpack_w4(w4)
    return (u - 8) * per_column(scale, u.shape[1])


def activations_fp8(codes, scale):
    return O.e4m3_decode(codes) * per_column(scale, codes.shape[1])


def read_kv_fp8(c8, scale, kr_bits, page_table, kv_lens, b):
    """The rows [kv_len, 576] of sequence b, unrounded."""
    n = int(kv_lens[b])
    c, kr = O.gather_sequence_fp8(c8, scale, kr_bits, page_table[b], n)
    return np.concatenate([c, kr], 1)
