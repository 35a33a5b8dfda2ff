"""The few-bit operators without a GPU: pins of their plain float64 definitions, and
the arguments their entry points refuse before touching the device."""

import ctypes

import numpy as np
import pytest
import torch

from oracle import few_bits_oracle as F
from oracle import mla_oracle as O

P, I, I64, FL = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float
OK, INVALID, UNSUPPORTED = 0, 1, 2


# ------------------------------------------------------------------ the definitions
def test_norm_definition_against_loops():
    rng = np.random.default_rng(0)
    x, r, w = rng.normal(size=(3, 24)), rng.normal(size=(3, 24)), rng.normal(size=24)
    h, v = F.rms_norm(x, w, 1e-3, r)
    for t in range(3):
        mean = sum((x[t, i] + r[t, i]) ** 2 for i in range(24)) / 24
        for i in range(24):
            assert abs(v[t, i] - (x[t, i] + r[t, i]) / (mean + 1e-3) ** 0.5 * w[i]) < 1e-12
    # a row of one magnitude has norm 1: v is its signs (eps = 0), whatever the magnitude
    for a in (1e-3, 7.0):
        assert np.allclose(F.rms_norm(np.full((1, 8), -a), np.ones(8), 0.0)[1], -1.0, atol=1e-14)
    assert np.array_equal(h, x + r)


def test_norm_scale_maps_the_largest_value_to_448():
    v = np.zeros((2, 200))
    v[0, 5], v[0, 150], v[1, 199] = -3.5, 448.0, 7.0
    s = F.norm_scale(v)
    assert s.shape == (2, 2)
    assert s[0, 0] == 3.5 / 448 and s[0, 1] == 1.0 and s[1, 0] == 2.0 ** -100 and s[1, 1] == 7.0 / 448


def test_bf16_round_equals_torch():
    v = np.random.default_rng(1).normal(size=4096) * np.exp2(np.random.default_rng(2).integers(-60, 60, 4096))
    ties = np.array([1.00390625, 1.01171875, -1.00390625, 257.0, 259.0, 0.0])  # halfway between neighbours
    v = np.concatenate([v.astype(np.float32).astype(np.float64), ties])
    ref = torch.tensor(v, dtype=torch.float32).to(torch.bfloat16).double().numpy()
    assert np.array_equal(F.bf16_round(v), ref)


def test_w4_format():
    u = np.arange(16).reshape(1, 16).repeat(4, 0)
    u = np.concatenate([u] * 4, 1)  # [4, 64]
    b = F.pack_w4(u)
    assert b.shape == (4, 32) and b[0, 0] == 0x10 and b[0, 7] == 0xfe
    assert np.array_equal(F.unpack_w4(b), u)
    s = np.full((4, 1), 0.5)
    assert F.weights_w4(b, s)[0, :4].tolist() == [-4.0, -3.5, -3.0, -2.5]
    assert F.weights_w4(b, s)[3, 15] == 3.5


def test_w4_quantiser_is_a_nearest_choice():
    rng = np.random.default_rng(3)
    w = F.bf16_round(rng.normal(size=(5, 192)) * np.exp2(rng.integers(-20, 20, (5, 1))))
    w[2] = 0.0
    u, s = F.quantize_w4(w)
    assert u.min() >= 0 and u.max() <= 15 and s.shape == (5, 2)
    assert np.array_equal(s[2], [1.0, 1.0]) and (u[2] == 8).all()
    back = F.weights_w4(F.pack_w4(u), s)
    # no other code comes nearer, and the largest weight of a group takes +-7
    col = F.per_column(s, 192)
    for c in range(-8, 8):
        assert (np.abs(w - back) <= np.abs(w - c * col) + 1e-30).all()
    assert (np.abs(u - 8).max(1) == [7, 7, 0, 7, 7]).all()


def test_w4_quantiser_has_no_near_ties_in_fp32():
    """The quotient of two bf16 values is a tie exactly or at least 2^-18 (relative) away from one, so rounding
    it to fp32 first cannot change the code; here for every pair of significands."""
    a = np.arange(128, 256, dtype=np.float64)
    for e in range(-4, 5):
        q = (a[:, None] * 2.0 ** e) / a[None, :]
        q = q[q <= 8.5]
        assert np.array_equal(np.rint(q), np.rint(q.astype(np.float32).astype(np.float64)))
    t = a / 7.0  # the scale: max / 7 is never near a tie between bf16 neighbours either
    assert np.array_equal(F.bf16_round(t), F.bf16_round(t.astype(np.float32).astype(np.float64)))


def test_read_definition():
    rng = np.random.default_rng(4)
    c8 = rng.integers(0, 0x7f, (3, 64, 512)).astype(np.uint8)
    s = rng.uniform(0.5, 2, (3, 64)).astype(np.float32)
    kr = rng.normal(size=(3, 64, 64)).astype(np.float16)
    rows = F.read_kv_fp8(c8, s, kr.view(np.uint16), np.array([[2, 0, -1]]), [70], 0)
    assert rows.shape == (70, 576)
    assert rows[69, 3] == float(s[0, 5]) * O.e4m3_decode(c8[0, 5, 3]) and rows[1, 512] == float(s[2, 1]) * float(kr[2, 1, 0])


# ------------------------------------------------------------------ refusals
@pytest.fixture(scope="module")
def lib():
    from mla_absorbed_decode_absorb_gb300 import build
    lib = ctypes.CDLL(build.build())
    lib.mla_rms_norm.argtypes = [P, I64, P, P, P, FL, P, P, P, I, I, P]
    lib.mla_quantize_w4.argtypes = [P, P, P, I, I, P]
    lib.mla_dequantize_w4.argtypes = [P, P, P, I, I, P]
    lib.mla_linear_w4.argtypes = [P, P, P, P, I, I, I, P]
    lib.mla_linear_w4_fp8.argtypes = [P, P, P, P, P, I, I, I, P]
    lib.mla_linear_w4_pair.argtypes = [P, I, I, P, P, I, P, P, P, I, P, P]
    lib.mla_linear_w4_fp8_pair.argtypes = [P, P, I, I, P, P, I, P, P, P, I, P, P]
    lib.mla_read_kv_fp8.argtypes = [P, P, P, I64, P, I, P, I, I, P, P]
    return lib


def at(i):
    """Addresses far apart, 16-byte aligned, never dereferenced (every call below is refused)."""
    return (i + 1) << 32


def test_rms_norm_refusals(lib):
    good = dict(x=at(0), x_ld=512, r=at(1), ro=at(2), w=at(3), eps=1e-6, y=at(4), y8=at(5), s=at(6), T=4, D=512)

    def call(**kw):
        a = {**good, **kw}
        return lib.mla_rms_norm(a["x"], a["x_ld"], a["r"], a["ro"], a["w"], a["eps"], a["y"], a["y8"], a["s"], a["T"],
                                a["D"], None)

    assert call(T=0) == OK
    for bad in [dict(T=-1), dict(D=0), dict(D=12), dict(x_ld=504), dict(x_ld=516), dict(eps=-1.0),
                dict(eps=float("nan")), dict(x=None), dict(w=None), dict(r=None), dict(ro=None), dict(y8=None),
                dict(s=None), dict(y=None, y8=None, s=None), dict(x=at(0) + 2), dict(r=at(1) + 8), dict(w=at(3) + 8),
                dict(y=at(4) + 2), dict(y8=at(5) + 8), dict(s=at(6) + 4),
                dict(ro=at(0)), dict(ro=at(1) + 512), dict(y=at(1)), dict(y=at(0) + 1024), dict(y=at(2)),
                dict(y8=at(4) + 512), dict(y8=at(0)), dict(s=at(3)),
                dict(y=at(0), x_ld=520)]:  # in place only with dense rows
        assert call(**bad) == INVALID, bad
    assert call(D=16392, x_ld=16392) == UNSUPPORTED


def test_w4_refusals(lib):
    for f in (lib.mla_quantize_w4, lib.mla_dequantize_w4):
        assert f(at(0), at(1), at(2), 0, 128, None) == INVALID
        assert f(at(0), at(1), at(2), 4, 96, None) == INVALID
        assert f(at(0), at(1), at(2), 4, 0, None) == INVALID
        assert f(at(0), at(1), at(2), 2 ** 30, 512, None) == UNSUPPORTED  # 2^32 groups
        assert f(at(0), at(1), at(2), 1, 2 ** 31 - 64, None) == UNSUPPORTED
        assert f(at(0), at(1), at(2), 2 ** 31 - 1, 64, None) == UNSUPPORTED
        for i in range(3):
            for bad in (None, at(i) + 8):
                a = [at(0), at(1), at(2)]
                a[i] = bad
                assert f(*a, 4, 128, None) == INVALID, (i, bad)
    assert lib.mla_quantize_w4(at(0), at(0) + 512, at(2), 4, 128, None) == INVALID     # codes inside w
    assert lib.mla_dequantize_w4(at(0), at(1), at(0) + 128, 4, 128, None) == INVALID   # w over the codes
    x, w4, s, y = at(0), at(1), at(2), at(3)
    for T, K, N in [(0, 128, 4), (257, 128, 4), (1, 96, 4), (1, 0, 4), (1, 128, 0)]:
        assert lib.mla_linear_w4(x, w4, s, y, T, K, N, None) == INVALID
        assert lib.mla_linear_w4_fp8(x, at(4), w4, s, y, T, K, N, None) == INVALID
    for a in [(None, w4, s, y), (x, None, s, y), (x, w4, None, y), (x, w4, s, None), (x + 8, w4, s, y),
              (x, w4 + 8, s, y), (x, w4, s + 8, y), (x, w4, s, y + 1), (x, w4, s, x + 64), (x, w4, s, w4)]:
        assert lib.mla_linear_w4(*a, 2, 128, 4, None) == INVALID, a
    assert lib.mla_linear_w4_fp8(x, None, w4, s, y, 2, 128, 4, None) == INVALID
    assert lib.mla_linear_w4_fp8(x, at(4) + 4, w4, s, y, 2, 128, 4, None) == INVALID
    assert lib.mla_linear_w4_fp8(x, y + 4, w4, s, y, 2, 128, 4, None) == INVALID
    for K, N in [(4194304 + 64, 4), (2 ** 31 - 64, 4), (64, 2 ** 30 + 1), (64, 2 ** 31 - 1)]:
        assert lib.mla_linear_w4(0x1000, 1 << 60, 1 << 61, 1 << 62, 1, K, N, None) == UNSUPPORTED
    good = [x, 2, 128, w4, s, 4, y, at(5), at(6), 6, at(7), None]
    for i, bad in [(0, None), (1, 0), (1, 257), (2, 96), (3, None), (4, None), (5, 0), (6, None), (7, None), (8, None),
                   (9, 0), (10, None), (0, x + 8), (3, w4 + 8), (7, at(5) + 8), (8, at(6) + 8), (10, at(7) + 1),
                   (10, y + 8), (6, at(5)), (10, w4), (10, x), (6, at(6))]:
        a = list(good)
        a[i] = bad
        assert lib.mla_linear_w4_pair(*a) == INVALID, (i, bad)
        assert lib.mla_linear_w4_fp8_pair(a[0], at(9), *a[1:]) == INVALID, (i, bad)
    assert lib.mla_linear_w4_fp8_pair(good[0], None, *good[1:]) == INVALID
    assert lib.mla_linear_w4_fp8_pair(good[0], y, *good[1:]) == INVALID


def test_read_refusals(lib):
    good = [at(0), at(1), at(2), 4, at(3), 2, at(4), 3, 128, at(5), None]

    def call(**kw):
        a = list(good)
        for i, v in kw.items():
            a[int(i[1:])] = v
        return lib.mla_read_kv_fp8(*a)

    assert call(a7=0) == OK and call(a8=0) == OK  # nothing to read
    for bad in [dict(a7=-1), dict(a8=-1), dict(a3=-1), dict(a5=-1), dict(a5=1), dict(a8=129)] + \
            [{f"a{i}": None} for i in (0, 1, 2, 4, 6, 9)] + [{f"a{i}": at(7) + 8} for i in (0, 1, 2, 9)]:
        assert call(**bad) == INVALID, bad
    assert call(a7=65536) == UNSUPPORTED
