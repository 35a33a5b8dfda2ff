"""Attention over the FP8 cache where a row's weights, its tokens' scales or its query's two parts span many powers of two,
against the plain float64 definition on the values that the cache stands for.

Tolerances.  A weight times its token's scale is rounded to 8 bits down to 2^-11 of the row's largest one (half a step,
2^-8 of it, uniform at the worst: 2^-8 / sqrt(3) = 2.3e-3 rms), and the output likewise: 3.2e-3, and the repository's
5e-3 for a head by itself, relative L2 of its O' and of its outputs.  Smaller weights have 3 bits down to 2^-26 (2^-3 /
sqrt(3) = 0.072 rms of each, signs at random).  Where n tokens share the weight, their sum is off by 0.072 / sqrt(n): 8e-4
for 8191 of them, 4.8e-3 at six deviations: 5e-3 again."""

import numpy as np
import pytest
import torch

from oracle import view_oracle as V
from test_gpu_view import PAGE, Problem, clean_status, f64  # noqa: F401

pytestmark = pytest.mark.gpu

HEADS = [0, 1, 37, 63, 64, 90, 127]


def fill(p, b, c, k, scale=None):
    """Sequence b's latent values c [T, 512] and rotated keys k [T, 64] into the FP8 cache, and what it then stands for."""
    s = c.abs().amax(1) / 448.0 if scale is None else scale
    code, key = (c / s[:, None]).to(torch.float8_e4m3fn), (k / s[:, None]).to(torch.float16)
    t = torch.arange(len(c))
    at = (p.table[b, t // PAGE].long(), t % PAGE)
    p.parts[0][at], p.parts[1][at], p.parts[2][at] = code.view(torch.uint8), s, key
    p.rows[b] = torch.cat([code.double() * s.double()[:, None], key.double() * s.double()[:, None]], 1).numpy()


def check(p, window=0, lse_tol=1.5e-3):
    """Each head's O' (one split) and outputs (one, and more), relative to the head's own norm."""
    seen = [V.visible(L, p.n_q, window) for L in p.prior]
    w = f64(p.w_uv)[HEADS]
    for split in (1 << 20, 3):
        out, lse, latent = p.run(split, window)
        for b in range(p.B):
            o_ref, lse_ref = V.attend(f64(p.q[b])[:, HEADS], p.rows[b], seen[b])
            assert np.abs(f64(lse[b])[:, HEADS] - lse_ref).max() < lse_tol
            ref = np.einsum("nhm,hdm->nhd", o_ref, w)
            err, size = np.linalg.norm(f64(out[b])[:, HEADS] - ref, axis=-1), np.linalg.norm(ref, axis=-1)
            assert (err <= 5e-3 * size).all(), (split, err, size)
            if p.splits == 1:
                err, size = np.linalg.norm(f64(latent[b])[:, HEADS] - o_ref, axis=-1), np.linalg.norm(o_ref, axis=-1)
                assert (err <= 5e-3 * size).all(), (err, size)


@pytest.mark.parametrize("shift", [0, 7, 9, 13, 16])
def test_large_scales_with_low_scores(shift):
    """Tokens whose scale is 2^shift times the others' and whose score is 37 nats lower weigh nothing, and take nothing
    from the others' weights."""
    p = Problem([200, 70], 2, seed=shift, fp8=True)
    g = torch.Generator().manual_seed(shift)
    for b in range(p.B):
        n = p.prior[b] + p.n_q
        c, k = torch.randn(n, 512, generator=g), torch.randn(n, 64, generator=g)
        c[:, 511], k[:, 0] = 0.0, 0.0
        s = c.abs().amax(1) / 448.0
        far = torch.arange(n) % 7 == 3
        c[far], k[far], s[far] = 0.0, 0.0, 2.0 ** (shift - 7)
        c[far, 511], k[far, 0] = 448.0 * 2.0 ** (shift - 7), -64.0
        fill(p, b, c, k, s)
    p.q[..., 511], p.q[..., 512] = 0.0, 8.0  # 8 x -64 / sqrt(192) = -37
    check(p)


@pytest.mark.parametrize("first", [1.0, 0.1])
def test_many_weak_tokens_behind_a_strong_one(first):
    """A first token that outweighs each other one by 8 to 17 nats (a head each), over values that share a mean: the weak
    ones' sum counts, and what a kernel loses of it does not cancel."""
    p = Problem([8191], 1, seed=1, fp8=True)
    g = torch.Generator().manual_seed(2)
    c, k = 1.0 + 0.3 * torch.randn(8192, 512, generator=g), torch.zeros(8192, 64)
    k[:, 0] = -(1.0 + 0.05 * torch.randn(8192, generator=g))
    c[0], k[0] = first, 0.0
    fill(p, 0, c, k)
    lat = torch.randn(128, 512, generator=g) * 0.226
    p.q[0, 0, :, :512] = (lat - lat.mean(1, keepdim=True)).to(torch.bfloat16)
    p.q[0, 0, :, 512:] = 0.0
    p.q[0, 0, :, 512] = (torch.linspace(8.0, 17.0, 128) * 192 ** 0.5).to(torch.bfloat16)
    # |q| |row| <= 236 x 1.2 + 6 x 24: 430, against 576 in the plain inputs
    check(p)


@pytest.mark.parametrize("x", [0, 4, 8, 12])
def test_a_query_whose_parts_differ_in_size(x):
    """Latent columns 2^x times smaller and rotated ones 2^x times larger, over rows the other way round: scores as ever,
    of which each part has half."""
    p = Problem([300, 64], 2, seed=x, fp8=True)
    g = torch.Generator().manual_seed(x)
    for b in range(p.B):
        n = p.prior[b] + p.n_q
        fill(p, b, torch.randn(n, 512, generator=g) * 2.0 ** x, torch.randn(n, 64, generator=g) * 2.0 ** -x)
    p.q[..., :512] *= 2.0 ** -x
    p.q[..., 512:] *= 2.0 ** x
    p.w_uv = (p.w_uv.float() * 2.0 ** -x).to(torch.bfloat16)
    check(p)


@pytest.mark.parametrize("zeros", [1, 64, 128, 300])
def test_tokens_of_scale_zero_count_in_the_sum(zeros):
    """A row of zeros with a scale of 0 is a token: score 0, value 0.  In front of the others, and alone."""
    p = Problem([400, max(zeros - 2, 0)], 2, seed=zeros, fp8=True)
    g = torch.Generator().manual_seed(zeros)
    for b in range(p.B):
        n = p.prior[b] + p.n_q
        c, k = torch.randn(n, 512, generator=g), torch.randn(n, 64, generator=g)
        s = c.abs().amax(1) / 448.0
        none = torch.arange(n) < zeros
        fill(p, b, torch.where(none[:, None], torch.zeros(()), c), torch.where(none[:, None], torch.zeros(()), k),
             torch.where(none, torch.ones(()), s))
        t = torch.arange(n)[none]
        p.parts[1][p.table[b, t // PAGE].long(), t % PAGE] = 0.0
    if zeros > 2:  # the second sequence holds nothing else: O' = 0, and the logarithm of the number of tokens
        out, lse, latent = p.run(1 << 20)
        n = torch.arange(1, 3) + p.prior[1]
        assert not latent[1].any() and not out[1].any()
        assert (lse[1].cpu() - n.float().log()[:, None]).abs().max() < 1e-5
        p.prior, p.B, p.table, p.q, p.rows = p.prior[:1], 1, p.table[:1], p.q[:1], p.rows[:1]
    check(p)
