"""The few-bit operators through the C ABI against their plain float64 definitions.

Tolerances, from the roundings each operator makes (half a step: bf16 2^-8,
E4M3 2^-4, fp32 2^-24 relative):

* norm: h = x + r is one fp32 sum, so r_out is within (2^-8 + 2^-24) |h|.  v passes
  the sum of D squares (at most D + 1 roundings, halved by the square root), the
  mean, eps, root, reciprocal, and two products: relative (D / 2 + 8) 2^-24 at
  most, then one bf16 rounding; in 8 bits a half step of E4M3 (2^-4 of the value,
  or 2^-10 of the scale below its normal range) instead.
* linear: products are exact, K of them and three operations per group in fp32
  (2^-23 of the summed magnitudes each, as for mla_linear), then one bf16 rounding.
* 4-bit weights: the same codes and scales; read back: one fp32 product, one bf16
  rounding.
* cache read back: bf16(fp32(s code)), bit for bit.
"""

import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from oracle import few_bits_oracle as F
from oracle import mla_oracle as O
from test_gpu_parity import bits

pytestmark = pytest.mark.gpu


def f64(t):
    return O.bf16_bits_to_f64(bits(t))


def ok():
    from mla_absorbed_decode_absorb_gb300 import ops
    torch.cuda.synchronize()
    assert ops.mla_get_device_status() == ops.MLA_OK


def within(got, ref, tol):
    got, ref = np.asarray(got, np.float64), np.asarray(ref, np.float64)
    assert np.isfinite(got).all()
    assert (np.abs(got - ref) <= tol).all(), float((np.abs(got - ref) - tol).max())


# ------------------------------------------------------------------ norm
def norm_inputs(T, D, seed, ld=None, residual=True):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, ld or D, generator=g).to(torch.bfloat16)
    r = (torch.randn(T, D, generator=g) * torch.where(torch.rand(D, generator=g) < 0.02, 30.0, 1.0)).to(torch.bfloat16)
    w = (1 + 0.2 * torch.randn(D, generator=g)).to(torch.bfloat16)
    return x.cuda()[:, :D], (r.cuda() if residual else None), w.cuda()


def check_norm(x, r, w, eps, r_out=None, y=None, y8=None, scale=None):
    D = x.shape[1]
    h, v = F.rms_norm(f64(x), f64(w), eps, None if r is None else f64(r))
    rel = (D / 2 + 8) * 2.0 ** -24
    if r_out is not None:
        within(f64(r_out), h, (2.0 ** -8 + 2.0 ** -24) * np.abs(h))
    if y is not None:
        within(f64(y), v, (2.0 ** -8 + 2 * rel) * np.abs(v))
    if y8 is not None:
        s_ref = F.norm_scale(v)
        s = scale.double().cpu().numpy()
        within(s, s_ref, (rel + 2.0 ** -23) * s_ref)
        col = F.per_column(s, D)
        value = O.e4m3_decode(y8.cpu().numpy()) * col
        within(value, v, np.maximum(2.0 ** -4 * np.abs(v), 2.0 ** -10 * col) + 3 * rel * np.abs(v))


@pytest.mark.parametrize("T,D", [(1, 8), (1, 7168), (3, 120), (2, 128), (5, 1544), (33, 1536), (130, 136), (64, 512),
                                 (2, 8192), (3, 8200), (2, 16384)])
@pytest.mark.parametrize("residual", [False, True])
def test_norm_parity(T, D, residual):
    from mla_absorbed_decode_absorb_gb300 import ops
    x, r, w = norm_inputs(T, D, T + D, residual=residual)
    out = torch.empty_like(x) if residual else None
    y = ops.mla_rms_norm(x, w, 1e-6, r, out)
    check_norm(x, r, w, 1e-6, r_out=out, y=y)
    y8, s = ops.mla_rms_norm_fp8(x, w, 1e-6, r, out)
    check_norm(x, r, w, 1e-6, r_out=out, y8=y8, scale=s)
    both = torch.empty(T, D, dtype=torch.bfloat16, device="cuda")
    z8, z = ops.mla_rms_norm_fp8(x, w, 1e-6, r, out, y=both)  # both forms at once
    assert torch.equal(z8, y8) and torch.equal(z, s) and torch.equal(both.view(torch.int16), y.view(torch.int16))
    ok()


def test_norm_reads_strided_rows():
    from mla_absorbed_decode_absorb_gb300 import ops
    x, r, w = norm_inputs(7, 512, 5, ld=576)
    assert not x.is_contiguous()
    check_norm(x, r, w, 1e-5, y=ops.mla_rms_norm(x, w, 1e-5, r, torch.empty_like(r)))
    one = x[:1]
    check_norm(one, None, w, 1e-5, y=ops.mla_rms_norm(one, w, 1e-5))
    ok()


def test_norm_in_place():
    from mla_absorbed_decode_absorb_gb300 import ops
    x, r, w = norm_inputs(9, 1536, 6)
    x = x.contiguous()
    x0, r0 = x.clone(), r.clone()
    ref_out = torch.empty_like(r)
    ref = ops.mla_rms_norm(x, w, 1e-6, r, ref_out)
    y = ops.mla_rms_norm(x, w, 1e-6, r, y=x)  # the residual in place (the default), y over x
    assert y.data_ptr() == x.data_ptr()
    assert torch.equal(y.view(torch.int16), ref.view(torch.int16))
    assert torch.equal(r.view(torch.int16), ref_out.view(torch.int16))
    check_norm(x0, r0, w, 1e-6, r_out=r, y=x)
    ok()


def test_norm_rows_of_zeros_and_non_finite_rows():
    """A zero row gives zeros (eps > 0) and NaN for eps = 0, as 0 * inf does; a NaN or an infinity makes its
    own row NaN and no other, in both forms."""
    from mla_absorbed_decode_absorb_gb300 import ops
    x, _, w = norm_inputs(6, 384, 8)
    x[1] = 0
    x[3, 200], x[4, 7] = float("nan"), float("-inf")
    y = ops.mla_rms_norm(x, w, 1e-6)
    y8, s = ops.mla_rms_norm_fp8(x, w, 1e-6)
    fine = [0, 1, 2, 5]
    check_norm(x[fine], None, w, 1e-6, y=y[fine], y8=y8[fine], scale=s[fine])
    assert (s[1] == 2.0 ** -100).all() and (y8[1] & 0x7f == 0).all()
    assert torch.isnan(y[3]).all() and (y8[3] & 0x7f == 0x7f).all()
    assert torch.isnan(y[4, 7]) and (y8[4, 7] & 0x7f) == 0x7f
    assert torch.isfinite(s[[0, 1, 2, 3, 5]]).all()
    z = ops.mla_rms_norm(x, w, 0.0)
    assert torch.isnan(z[1]).all() and torch.isfinite(z[fine[2:]].float()).all()
    ok()


@pytest.mark.parametrize("xe,we", [(-50, -80), (-50, 100), (50, -100), (50, 100), (0, -100), (0, 120)])
def test_norm_of_small_and_large_values(xe, we):
    """Rows of about 2^xe times a weight of about 2^we, whose product may leave fp32's range where v does not: v in
    both forms, and the scale's floor of 2^-100 below it."""
    from mla_absorbed_decode_absorb_gb300 import ops
    x, r, w = norm_inputs(5, 384, 77)
    x, r, w = x * 2.0 ** xe, r * 2.0 ** xe, w * 2.0 ** we
    x[:, 5], r[:, 5] = 0, 0
    for res in (None, r):
        out = None if res is None else torch.empty_like(res)
        check_norm(x, res, w, 0.0, r_out=out, y=ops.mla_rms_norm(x, w, 0.0, res, out))
        y8, s = ops.mla_rms_norm_fp8(x, w, 0.0, res, out)
        check_norm(x, res, w, 0.0, y8=y8, scale=s)
    ok()


def test_norm_of_no_rows_and_refusals():
    from mla_absorbed_decode_absorb_gb300 import ops
    x, r, w = norm_inputs(4, 256, 9)
    assert ops.mla_rms_norm(x[:0], w).shape == (0, 256)
    with pytest.raises(ops.MLAError):
        ops.mla_rms_norm(torch.zeros(2, 12, dtype=torch.bfloat16, device="cuda"), w[:12])  # D not a multiple of 8
    with pytest.raises(ValueError):
        ops.mla_rms_norm(x.t(), w[:4].contiguous())   # columns not contiguous
    with pytest.raises(ValueError):
        ops.mla_rms_norm(x, w[:128].contiguous())     # weight of another width
    with pytest.raises(TypeError):
        ops.mla_rms_norm(x.float(), w)
    with pytest.raises(ValueError):
        ops.mla_rms_norm(x, w, residual_out=r)
    with pytest.raises(ops.MLAError):
        ops.mla_rms_norm(x, w, residual=r, y=r)       # y over the residual
    ok()


# ------------------------------------------------------------------ 4-bit weights
@pytest.mark.parametrize("N,K", [(1, 64), (1, 128), (3, 192), (17, 1600), (64, 7168), (577, 704), (130, 64)])
def test_quantize_and_dequantize_w4(N, K):
    from mla_absorbed_decode_absorb_gb300 import ops
    g = torch.Generator().manual_seed(N + K)
    w = (torch.randn(N, K, generator=g) * torch.exp2(torch.randint(-9, 4, (N, 1), generator=g).float()))
    w = w.to(torch.bfloat16)
    w[0, :64] = 0
    u, s = F.quantize_w4(f64(w))
    w4, scale = ops.mla_quantize_w4(w.cuda())
    assert np.array_equal(w4.cpu().numpy(), F.pack_w4(u))
    assert np.array_equal(f64(scale), s)
    back = ops.mla_dequantize_w4(w4, scale)
    ref = F.weights_w4(F.pack_w4(u), s)
    within(f64(back), ref, (2.0 ** -8) * np.abs(ref))
    assert np.array_equal(f64(back), F.bf16_round(ref))  # (u - 8) s has 12 bits: exact in fp32
    ok()


def test_quantize_w4_of_the_smallest_weights():
    """max / 7 below bf16's smallest value: the scale is 1 and the codes are zeros."""
    from mla_absorbed_decode_absorb_gb300 import ops
    w = torch.full((2, 128), 2.0 ** -133, dtype=torch.bfloat16, device="cuda")
    w[1] = -0.0
    w4, s = ops.mla_quantize_w4(w)
    assert (w4 == 0x88).all() and (s == 1).all()
    ok()


# ------------------------------------------------------------------ linear
def linear_inputs(T, K, N, fp8, seed):
    rng = np.random.default_rng(seed)
    w4 = rng.integers(0, 256, (N, K // 2)).astype(np.uint8)
    scale = torch.tensor(rng.uniform(0.5, 1.5, (N, F.groups(K))) / (4.6 * K ** 0.5)).to(torch.bfloat16)
    if fp8:
        x = rng.integers(0, 256, (T, K)).astype(np.uint8)
        x[(x & 0x7f) == 0x7f] = 0
        x = torch.tensor(x)
        sx = torch.tensor(rng.uniform(0.5, 2.0, (T, F.groups(K))) / 200, dtype=torch.float32)
    else:
        x, sx = torch.tensor(rng.normal(size=(T, K))).to(torch.bfloat16), None
    return x, sx, torch.tensor(w4), scale


def linear_ref(x, sx, w4, scale):
    xf = f64(x) if sx is None else F.activations_fp8(x.numpy(), sx.double().numpy())
    wf = F.weights_w4(w4.numpy(), f64(scale))
    ref, mag = xf @ wf.T, np.abs(xf) @ np.abs(wf).T
    K = xf.shape[1]
    return ref, 2.0 ** -8 * np.abs(ref) + (K + 3 * F.groups(K)) * 2.0 ** -23 * mag + 1e-30


def run_linear(x, sx, w4, scale, **kw):
    from mla_absorbed_decode_absorb_gb300 import ops
    if sx is None:
        return ops.mla_linear_w4(x.cuda(), w4.cuda(), scale.cuda(), **kw)
    return ops.mla_linear_w4_fp8(x.cuda(), sx.cuda(), w4.cuda(), scale.cuda(), **kw)


@pytest.mark.parametrize("T,K,N", [
    (1, 64, 1), (1, 128, 16), (1, 7168, 64), (1, 16384, 130), (2, 192, 15), (3, 1600, 577), (7, 320, 63), (8, 1024, 65),
    (9, 1088, 200), (16, 7168, 576), (17, 64, 129), (24, 2112, 40), (31, 1536, 300), (32, 1536, 2048), (33, 448, 128),
    (64, 1536, 1000), (65, 704, 257), (100, 7168, 144), (128, 512, 384), (129, 192, 127), (200, 1152, 640),
    (255, 640, 96), (256, 7104, 577)])
@pytest.mark.parametrize("fp8", [False, True])
def test_linear_parity(T, K, N, fp8):
    args = linear_inputs(T, K, N, fp8, T * 131 + K + N)
    ref, tol = linear_ref(*args)
    y = run_linear(*args)
    within(f64(y), ref, tol)
    again = run_linear(*args)  # K is summed in a fixed order
    assert torch.equal(y.view(torch.int16), again.view(torch.int16))
    ok()


# Sizes of over 36 M weights times passes of 8 tokens: the tensor-core kernel, its tiles of 16, 48, 64 and 128 tokens
# each full and ragged, K of one group, half a group and not a multiple of 128, odd widths, K whole and divided.
@pytest.mark.parametrize("T,K,N", [
    (9, 1088, 16601), (16, 192, 94000), (16, 7168, 2561), (17, 64, 188001), (33, 1536, 4703), (48, 128, 47000),
    (49, 320, 16100), (57, 2112, 2200), (64, 1536, 3001), (65, 64, 62600), (100, 1088, 2600), (128, 128, 17600),
    (129, 576, 3700), (200, 1600, 901), (256, 64, 17700), (256, 16384, 130)])
@pytest.mark.parametrize("fp8", [False, True])
def test_linear_parity_large(T, K, N, fp8):
    assert N * K * -(-T // 8) > 36_000_000
    args = linear_inputs(T, K, N, fp8, T * 131 + K + N)
    ref, tol = linear_ref(*args)
    y = run_linear(*args)
    within(f64(y), ref, tol)
    again = run_linear(*args)
    assert torch.equal(y.view(torch.int16), again.view(torch.int16))
    ok()


# More tiles of 128 tokens than fit the GPU at once or than fill it: clusters whose CTAs take parts of several tiles
# (tails, whole ones and heads), one and two slices of the tokens, K ragged and short.
@pytest.mark.parametrize("T,K,N", [(130, 8192, 7100), (256, 4160, 7168), (200, 7104, 12900), (100, 5184, 17000),
                                   (256, 1088, 20001), (65, 256, 60000), (192, 10240, 9600)])
@pytest.mark.parametrize("fp8", [False, True])
def test_linear_of_shared_tiles(T, K, N, fp8):
    args = linear_inputs(T, K, N, fp8, T * 131 + K + N)
    ref, tol = linear_ref(*args)
    buf = torch.full((T + 2, N), 77.0, dtype=torch.bfloat16, device="cuda")
    y = run_linear(*args, y=buf[1:T + 1])
    within(f64(y), ref, tol)
    assert (buf[0] == 77).all() and (buf[T + 1] == 77).all()
    again = run_linear(*args)
    assert torch.equal(y.view(torch.int16), again.view(torch.int16))
    ok()


@pytest.mark.parametrize("T,K,N0,N1", [(1, 7168, 512, 64), (3, 192, 17, 1), (8, 1088, 1, 700), (5, 128, 9000, 9001),
                                       (32, 1536, 5000, 2600), (16, 192, 50001, 47000), (64, 704, 3000, 5001),
                                       (100, 1088, 1300, 1301), (256, 64, 8000, 9700), (100, 4160, 5000, 9001),
                                       (140, 4160, 3700, 3601)])
@pytest.mark.parametrize("fp8", [False, True])
def test_linear_pair_parity(T, K, N0, N1, fp8):
    """Two projections of one x in one launch, in both kernels; the second one's rows stay its own."""
    from mla_absorbed_decode_absorb_gb300 import ops
    x, sx, w4, scale = linear_inputs(T, K, N0, fp8, T + K)
    _, _, w4b, scale_b = linear_inputs(T, K, N1, fp8, T + K + 1)
    w0, w1 = (w4.cuda(), scale.cuda()), (w4b.cuda(), scale_b.cuda())
    if fp8:
        y0, y1 = ops.mla_linear_w4_fp8_pair(x.cuda(), sx.cuda(), w0, w1)
    else:
        y0, y1 = ops.mla_linear_w4_pair(x.cuda(), w0, w1)
    for y, w, s in ((y0, w4, scale), (y1, w4b, scale_b)):
        ref, tol = linear_ref(x, sx, w, s)
        assert y.shape == ref.shape
        within(f64(y), ref, tol)
    ok()


@pytest.mark.parametrize("T,N", [(8, 500), (16, 150000), (48, 50000), (64, 36000), (256, 9300)])
def test_linear_keeps_what_cancels(T, N):
    """Pairs of columns with one x (2 .. 30) and weights c and -c, and one column of the smallest E4M3 value 2^-9,
    which is what remains.  A partial sum is a multiple of 2^-9 below 64 * 7 * 30 < 2^14: 23 bits, so nothing is
    rounded but y, in whatever order the sums are formed."""
    rng = np.random.default_rng(T)
    K = 128
    c = rng.integers(1, 8, (N, K // 2))
    u = np.empty((N, K), np.int64)
    u[:, 0::2], u[:, 1::2] = 8 + c, 8 - c
    codes = rng.integers(0x40, 0x60, (T, K // 2)).astype(np.uint8)  # 2 .. 30
    x = np.repeat(codes, 2, axis=1)
    x[:, 0], x[:, 1], u[:, 1] = 1, 1, 8
    perm = rng.permutation(K)
    u, x = np.ascontiguousarray(u[:, perm]), np.ascontiguousarray(x[:, perm])
    w4, scale = torch.tensor(F.pack_w4(u)), torch.ones(N, 1, dtype=torch.bfloat16)
    xf = O.e4m3_decode(x)
    ref = F.bf16_round(np.broadcast_to(2.0 ** -9 * c[:, 0], (T, N)))
    y8 = run_linear(torch.tensor(x), torch.ones(T, 1), w4, scale)
    assert np.array_equal(f64(y8), ref)
    y = run_linear(torch.tensor(xf).to(torch.bfloat16), None, w4, scale)
    assert np.array_equal(f64(y), ref)
    ok()


@pytest.mark.parametrize("T", [1, 5, 32, 48, 256])
@pytest.mark.parametrize("fp8", [False, True])
def test_linear_of_extreme_codes(T, fp8):
    """Every weight -8, then every weight 7 (the ends of the range), then 0; the sums are exact integers times
    the scales, and a row of scale 0 gives 0."""
    N, K = 70, 320
    check_extreme_codes(T, N, K, fp8)
    if T > 5:
        check_extreme_codes(T, 36_000_000 // (K * -(-T // 8)) + 71, K, fp8)  # ... and the tensor-core kernel


def check_extreme_codes(T, N, K, fp8):
    x, sx, w4, scale = linear_inputs(T, K, N, fp8, 3)
    scale[5] = 0
    for byte, v in ((0x00, -8), (0xff, 7), (0x88, 0)):
        w4[:] = byte
        ref, tol = linear_ref(x, sx, w4, scale)
        y = run_linear(x, sx, w4, scale)
        within(f64(y), ref, tol)
        assert (f64(y)[:, 5] == 0).all() and (v != 0 or (f64(y) == 0).all())
    ok()


@pytest.mark.parametrize("T,N", [(2, 100), (9, 100), (9, 32000), (40, 100), (40, 12600), (57, 8000), (130, 100),
                                 (130, 3700)])
@pytest.mark.parametrize("fp8", [False, True])
def test_linear_keeps_a_bad_token_to_itself(T, N, fp8):
    """A NaN in one token's input (its code 0x7F) makes that token's outputs NaN and leaves the others'."""
    x, sx, w4, scale = linear_inputs(T, 576, N, fp8, 11)
    good = run_linear(x, sx, w4, scale)
    x[1, 570] = 0x7f if fp8 else float("nan")
    y = run_linear(x, sx, w4, scale)
    assert torch.isnan(y[1]).all()
    keep = [t for t in range(T) if t != 1]
    assert torch.equal(y[keep].view(torch.int16), good[keep].view(torch.int16))
    ok()


@pytest.mark.parametrize("T,N", [(1, 37), (20, 37), (70, 37), (10, 70001), (20, 47001), (60, 17601), (70, 15701)])
def test_linear_writes_its_rows_only(T, N):
    """y in the middle of a larger buffer, at an odd row width (no alignment beyond an element's)."""
    x, sx, w4, scale = linear_inputs(T, 256, N, False, 21)
    buf = torch.full((T + 2, N), 77.0, dtype=torch.bfloat16, device="cuda")
    run_linear(x, sx, w4, scale, y=buf[1:T + 1])
    ref, tol = linear_ref(x, sx, w4, scale)
    within(f64(buf[1:T + 1]), ref, tol)
    assert (buf[0] == 77).all() and (buf[T + 1] == 77).all()
    ok()


@pytest.mark.parametrize("T,K,N", [(3, 512, 64), (20, 7168, 2048), (40, 7168, 1536), (100, 8192, 7168), (70, 262144, 3)])
def test_linear_into_a_row_of_no_alignment(T, K, N):
    """y two bytes off every larger boundary, at widths that a wider store would take."""
    args = linear_inputs(T, K, N, False, 22)
    buf = torch.full((T * N + 8,), 77.0, dtype=torch.bfloat16, device="cuda")
    y = buf[3:3 + T * N].view(T, N)
    run_linear(*args, y=y)
    ref, tol = linear_ref(*args)
    within(f64(y), ref, tol)
    assert (buf[:3] == 77).all() and (buf[3 + T * N:] == 77).all()
    ok()


def test_offsets_past_32_bits():
    """Weights of more than 2^32 values and 2^31 bytes, activations and caches of more than 2^31 elements: rows at the
    start, on both sides of the borders and at the end."""
    from mla_absorbed_decode_absorb_gb300 import ops
    N, K = 270000, 16384
    g = torch.Generator(device="cuda").manual_seed(5)
    w4 = torch.randint(0, 256, (N, K // 2), generator=g, dtype=torch.uint8, device="cuda")
    scale = (torch.rand(N, K // 128, generator=g, device="cuda") / 600 + 1e-3).to(torch.bfloat16)
    border = 2 ** 31 // (K // 2)
    rows = torch.tensor([0, 1, 2 ** 31 // K - 1, 2 ** 31 // K, border - 1, border, border + 1, N - 2, N - 1], device="cuda")
    ref_w = F.weights_w4(w4[rows].cpu().numpy(), f64(scale[rows].cpu()))
    for T in (2, 12, 100):
        x = torch.randn(T, K, generator=g, device="cuda").to(torch.bfloat16)
        y = ops.mla_linear_w4(x, w4, scale)
        xf = f64(x.cpu())
        ref, mag = xf @ ref_w.T, np.abs(xf) @ np.abs(ref_w).T
        within(f64(y[:, rows].cpu()), ref, 2.0 ** -8 * np.abs(ref) + (K + 3 * (K // 128)) * 2.0 ** -23 * mag)
        del y
    n = 2 ** 31 // K + 40  # weights of more than 2^31 elements there and back
    back = ops.mla_dequantize_w4(w4[:n], scale[:n])
    again, s2 = ops.mla_quantize_w4(back)
    rows = torch.tensor([0, n - 41, n - 40, n - 1], device="cuda")
    assert np.array_equal(f64(back[rows].cpu()), F.bf16_round(F.weights_w4(w4[rows].cpu().numpy(), f64(scale[rows].cpu()))))
    u, s_ref = F.quantize_w4(f64(back[rows].cpu()))
    assert np.array_equal(again[rows].cpu().numpy(), F.pack_w4(u)) and np.array_equal(f64(s2[rows].cpu()), s_ref)
    del w4, scale, again, s2
    # the norm of those rows, in place, and in 8 bits
    w = torch.ones(K, dtype=torch.bfloat16, device="cuda")
    before = back[rows].clone()
    y8, s8 = ops.mla_rms_norm_fp8(back, w)
    check_norm(before, None, w, 1e-6, y8=y8[rows], scale=s8[rows])
    del y8
    ops.mla_rms_norm(back, w, y=back)
    check_norm(before, None, w, 1e-6, y=back[rows])
    del back
    # a cache read back into more than 2^31 elements: every sequence the same pages
    B, most = 60, 64 * 1000 + 5
    c8, sc, kr, pt, _ = fp8_cache([64 * 1001], 6)
    cache, ptg, _ = to_gpu(c8, sc, kr, pt, np.zeros(1, np.int32))
    lens = torch.full((B,), most, dtype=torch.int32, device="cuda")
    rows = ops.mla_read_kv_fp8(cache, ptg.expand(B, -1).contiguous(), lens, most).view(B, 1001 * 64, 576)
    assert rows.numel() > 2 ** 31
    assert torch.equal(rows[-1, :most].view(torch.int16), rows[0, :most].view(torch.int16))
    assert torch.isnan(rows[-1, most:].float()).all()
    t = most - 1
    ref = O.f32_to_bf16_bits(O.e4m3_decode(c8[pt[0, t // 64], t % 64]).astype(np.float32) * sc[pt[0, t // 64], t % 64])
    assert np.array_equal(bits(rows[-1, t, :512]), ref)
    ok()


def test_linear_refusals():
    from mla_absorbed_decode_absorb_gb300 import ops
    x, _, w4, scale = (t if t is None else t.cuda() for t in linear_inputs(4, 256, 8, False, 1))
    with pytest.raises(ops.MLAError):
        ops.mla_linear_w4(torch.zeros(257, 256, dtype=torch.bfloat16, device="cuda"), w4, scale)
    with pytest.raises(ops.MLAError):
        ops.mla_linear_w4(torch.zeros(0, 256, dtype=torch.bfloat16, device="cuda"), w4, scale)
    with pytest.raises(ops.MLAError):
        ops.mla_quantize_w4(torch.zeros(4, 96, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError):
        ops.mla_linear_w4(x, w4[:, :64].contiguous(), scale)
    with pytest.raises(ValueError):
        ops.mla_linear_w4(x, w4, scale[:, :1].contiguous())
    with pytest.raises(ValueError):
        ops.mla_linear_w4(x.t().contiguous().t(), w4, scale)
    with pytest.raises(ValueError):
        ops.mla_linear_w4(x.cpu(), w4, scale)
    with pytest.raises(TypeError):
        ops.mla_linear_w4(x.half(), w4, scale)
    ok()


# ------------------------------------------------------------------ cache read back
def fp8_cache(lens, seed, extra_pages=0):
    rng = np.random.default_rng(seed)
    need = [-(-n // 64) for n in lens]
    pool = sum(need) + 3
    c8 = rng.integers(0, 256, (pool, 64, 512)).astype(np.uint8)
    c8[(c8 & 0x7f) == 0x7f] = 0
    scale = rng.uniform(2.0 ** -10, 3, (pool, 64)).astype(np.float32)
    kr = rng.normal(size=(pool, 64, 64)).astype(np.float16)
    perm = rng.permutation(pool)
    pt = np.full((len(lens), max(max(need), 1) + extra_pages), -1, np.int32)
    k = 0
    for b, n in enumerate(need):
        pt[b, :n] = perm[k:k + n]
        k += n
    return c8, scale, kr, pt, np.array(lens, np.int32)


def to_gpu(c8, scale, kr, pt, lens):
    return (torch.tensor(c8).cuda(), torch.tensor(scale).cuda(), torch.tensor(kr).cuda()), torch.tensor(pt).cuda(), \
        torch.tensor(lens).cuda()


@pytest.mark.parametrize("lens", [[1], [64], [65], [0, 1, 63, 64, 65, 200], [300], [0, 0], [1000, 7, 513]])
@pytest.mark.parametrize("slack", [0, 40])
def test_read_back_bit_exact(lens, slack):
    """bf16(fp32(s value)) for every token, and the rows past a sequence's length as they were."""
    from mla_absorbed_decode_absorb_gb300 import ops
    c8, scale, kr, pt, n = fp8_cache(lens, sum(lens) + slack, extra_pages=1)
    cache, ptg, ng = to_gpu(c8, scale, kr, pt, n)
    most = max(max(lens), 1) + slack
    pages = -(-most // 64)
    if pages > pt.shape[1]:
        pytest.skip("the page table has no such page")
    rows = torch.full((len(lens) * pages, 64, 576), 5.0, dtype=torch.bfloat16, device="cuda")
    assert ops.mla_read_kv_fp8(cache, ptg, ng, most, rows).data_ptr() == rows.data_ptr()
    got = bits(rows).reshape(len(lens), pages * 64, 576)
    five = int(bits(torch.tensor([5.0], dtype=torch.bfloat16))[0])
    for b, k in enumerate(lens):
        t = np.arange(k)
        page, slot = pt[b, t // 64], t % 64
        s = scale[page, slot][:, None]
        v = np.concatenate([O.e4m3_decode(c8[page, slot]).astype(np.float32) * s,
                            kr[page, slot].astype(np.float32) * s], 1)
        assert np.array_equal(got[b, :k], O.f32_to_bf16_bits(v))
        ref = F.read_kv_fp8(c8, scale, kr.view(np.uint16), pt, lens, b)
        within(O.bf16_bits_to_f64(got[b, :k]), ref, (2.0 ** -8 + 2.0 ** -24) * np.abs(ref) + 2.0 ** -126)
        assert (got[b, k:] == five).all()
    ok()


def test_read_back_skips_what_is_out_of_range():
    """A page id outside the pool loses that page, a length outside [0, max_kv_len] that sequence; the status
    says so and the rest is exact."""
    from mla_absorbed_decode_absorb_gb300 import ops
    c8, scale, kr, pt, n = fp8_cache([130, 100, 70, 64], 4)
    clean = ops.mla_read_kv_fp8(*to_gpu(c8, scale, kr, pt, n), 192)
    ok()
    pt2, n2 = pt.copy(), n.copy()
    pt2[0, 1] = c8.shape[0]
    n2[1], n2[2] = 193, -1
    rows = torch.zeros_like(clean)
    ops.mla_read_kv_fp8(*to_gpu(c8, scale, kr, pt2, n2), 192, rows)
    torch.cuda.synchronize()
    assert ops.mla_get_device_status() == ops.MLA_ERR_BOUNDS
    a, b = bits(rows).reshape(4, 3, 64, 576), bits(clean).reshape(4, 3, 64, 576)
    assert np.array_equal(a[0, 0], b[0, 0]) and np.array_equal(a[0, 2, :2], b[0, 2, :2]) and (a[0, 1] == 0).all()
    assert (a[1] == 0).all() and (a[2] == 0).all() and np.array_equal(a[3, 0], b[3, 0])
    ok()


# ------------------------------------------------------------------ how they are called
def chain(ops, x, r, w, w4, scale, out, y8, s, y):
    ops.mla_rms_norm_fp8(x, w, 1e-6, r, out, y8, s)
    ops.mla_linear_w4_fp8(y8, s, w4, scale, y)
    return y


@pytest.mark.parametrize("T,D,N", [(20, 1536, 600), (100, 4160, 9000)])
@pytest.mark.parametrize("overlap", [0, 1, 2])
def test_chain_on_a_side_stream_and_replayed(overlap, T, D, N):
    """Norm then projection on a stream of their own, then captured once and replayed on new inputs: the same
    bits as the calls one by one."""
    from mla_absorbed_decode_absorb_gb300 import ops
    before = ops.mla_get_launch_overlap()
    ops.mla_set_launch_overlap(overlap)
    try:
        x, r, w = norm_inputs(T, D, 31)
        x2, r2, _ = norm_inputs(T, D, 32)
        _, _, w4, scale = (t if t is None else t.cuda() for t in linear_inputs(T, D, N, False, 33))

        def fresh():
            return (torch.empty_like(x), torch.empty(T, D, dtype=torch.uint8, device="cuda"),
                    torch.empty(T, F.groups(D), dtype=torch.float32, device="cuda"),
                    torch.empty(T, N, dtype=torch.bfloat16, device="cuda"))

        ref = [chain(ops, a, b, w, w4, scale, *fresh()).clone() for a, b in ((x, r), (x2, r2))]
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        bufs = fresh()
        xin, rin = x.clone(), r.clone()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            y = chain(ops, xin, rin, w, w4, scale, *bufs)
        side.synchronize()
        assert torch.equal(y.view(torch.int16), ref[0].view(torch.int16))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            chain(ops, xin, rin, w, w4, scale, *bufs)
        for k, (a, b) in enumerate(((x, r), (x2, r2), (x, r))):
            xin.copy_(a), rin.copy_(b)
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(y.view(torch.int16), ref[k % 2].view(torch.int16))
        ok()
    finally:
        ops.mla_set_launch_overlap(before)


@pytest.mark.parametrize("overlap", [1, 2])
def test_projections_in_a_row_on_one_buffer(overlap):
    """y of one projection is x of the next, back to back through both kernels and into a buffer that the call before
    still reads: each call sees what came before it, eagerly and replayed."""
    from mla_absorbed_decode_absorb_gb300 import ops
    before = ops.mla_get_launch_overlap()
    ops.mla_set_launch_overlap(overlap)
    try:
        T, D = 96, 4096
        ws = [[t.cuda() for t in linear_inputs(T, D, D, False, 50 + i)[2:]] for i in range(3)]
        x0 = linear_inputs(T, D, 64, False, 60)[0].cuda()
        small = x0[:3].clone()

        def steps(a, b, c, d):
            for w in ws * 2:
                ops.mla_linear_w4(a, *w, b)
                ops.mla_linear_w4(b, *w, a)
                ops.mla_linear_w4(c, *w, d)
                ops.mla_linear_w4(d, *w, c)

        def slowly():
            a, c = x0.clone(), small.clone()
            for w in ws * 2:
                for _ in range(2):
                    a, c = ops.mla_linear_w4(a, *w), ops.mla_linear_w4(c, *w)
                    torch.cuda.synchronize()
            return a, c

        ref_a, ref_c = slowly()
        a, b, c, d = x0.clone(), torch.empty_like(x0), small.clone(), torch.empty_like(small)
        steps(a, b, c, d)
        assert torch.equal(a.view(torch.int16), ref_a.view(torch.int16))
        assert torch.equal(c.view(torch.int16), ref_c.view(torch.int16))
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            steps(a, b, c, d)
        for _ in range(3):
            a.copy_(x0), c.copy_(small)
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(a.view(torch.int16), ref_a.view(torch.int16))
            assert torch.equal(c.view(torch.int16), ref_c.view(torch.int16))
        ok()
    finally:
        ops.mla_set_launch_overlap(before)


def test_first_call_inside_a_capture():
    """A process whose first use of each kernel is captured: what the library asks the device for then is allowed."""
    code = """
import torch
from mla_absorbed_decode_absorb_gb300 import ops
g = torch.Generator(device="cuda").manual_seed(0)
w = torch.randn(9000, 4160, generator=g, device="cuda").to(torch.bfloat16)
xs = [torch.randn(t, 4160, generator=g, device="cuda").to(torch.bfloat16) for t in (1, 16, 40, 64, 200)]
gamma = torch.ones(4160, dtype=torch.bfloat16, device="cuda")
torch.cuda.synchronize()

def calls():
    w4, s = ops.mla_quantize_w4(w)
    out = []
    for x in xs:
        y8, ys = ops.mla_rms_norm_fp8(x, gamma)
        out += [ops.mla_linear_w4(x, w4, s), ops.mla_linear_w4_fp8(y8, ys, w4, s)]
    return out

graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = calls()
graph.replay()
torch.cuda.synchronize()
assert all(torch.equal(a.view(torch.int16), b.view(torch.int16)) for a, b in zip(got, calls()))
torch.cuda.synchronize()
assert ops.mla_get_device_status() == ops.MLA_OK
print("captured")
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]


def test_two_calls_at_once():
    """The same projection on two streams at once: no state is shared between calls."""
    from mla_absorbed_decode_absorb_gb300 import ops
    a = [t if t is None else t.cuda() for t in linear_inputs(6, 7168, 576, False, 41)]
    b = [t if t is None else t.cuda() for t in linear_inputs(40, 7168, 576, False, 42)]
    ra, rb = ops.mla_linear_w4(a[0], a[2], a[3]), ops.mla_linear_w4(b[0], b[2], b[3])
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    ya, yb = [torch.empty_like(ra) for _ in range(8)], [torch.empty_like(rb) for _ in range(8)]
    torch.cuda.synchronize()
    for i in range(8):
        ops.mla_linear_w4(a[0], a[2], a[3], ya[i], stream=s1)
        ops.mla_linear_w4(b[0], b[2], b[3], yb[i], stream=s2)
    ok()
    assert all(torch.equal(t.view(torch.int16), ra.view(torch.int16)) for t in ya)
    assert all(torch.equal(t.view(torch.int16), rb.view(torch.int16)) for t in yb)


def test_two_tensor_core_calls_at_once():
    """Clusters of two launches share SMs and their tensor memory: both finish, with the results of either alone.
    Up to 64 tokens a CTA holds 256 columns of its SM's tensor memory, beyond 512."""
    from mla_absorbed_decode_absorb_gb300 import ops
    shapes = ((40, 7168, 1536), (128, 7168, 577), (64, 16384, 900), (256, 7168, 576))
    args = [[t if t is None else t.cuda() for t in linear_inputs(T, K, N, False, T)] for T, K, N in shapes]
    ref = [ops.mla_linear_w4(a[0], a[2], a[3]) for a in args]
    streams = [torch.cuda.Stream() for _ in shapes]
    out = [[torch.empty_like(r) for _ in range(8)] for r in ref]
    torch.cuda.synchronize()
    for i in range(8):
        for a, y, s in zip(args, out, streams):
            ops.mla_linear_w4(a[0], a[2], a[3], y[i], stream=s)
    ok()
    for r, ys in zip(ref, out):
        assert all(torch.equal(y.view(torch.int16), r.view(torch.int16)) for y in ys)


def test_read_back_feeds_the_non_absorbed_path():
    """FP8 append, read back, decompress: keys and values of the dequantised cache rows."""
    from mla_absorbed_decode_absorb_gb300 import ops
    from mla_absorbed_decode_absorb_gb300 import workloads as W
    inp = W.generate(W.custom("read", [70, 5], n_q=3), seed=2)
    rope = ops.rope_table(100)
    cache = ops.fp8_cache_empty(inp.num_pages, "cuda")
    pt = inp.page_table.cuda()
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    for b in range(2):
        c, k = inp.sequence(b)
        ops.mla_append_kv_fp8(c.cuda()[None], k.cuda()[None], zero, pt[b:b + 1], rope, cache)
    lens = inp.kv_lens.cuda()
    rows = ops.mla_read_kv_fp8(cache, pt, lens, 73)
    ident = torch.arange(4, dtype=torch.int32, device="cuda").view(2, 2)
    k, v = ops.mla_decompress_kv(rows, ident, lens, 73, inp.w_uk.cuda(), inp.w_uv.cuda())
    for b in range(2):
        n = int(inp.kv_lens[b])
        c = f64(rows.view(2, 128, 576)[b, :n, :512])
        kd, vd = O.decompress_kv(c, f64(inp.w_uk), f64(inp.w_uv))
        km, vm = O.decompress_kv(np.abs(c), np.abs(f64(inp.w_uk)), np.abs(f64(inp.w_uv)))
        for got, ref, mag in ((k[b, :, :n], kd, km), (v[b, :, :n], vd, vm)):
            within(f64(got).transpose(1, 0, 2), ref, 2.0 ** -8 * np.abs(ref) + 512 * 2.0 ** -23 * mag)
    ok()
