"""The masked attention's roundings, each by itself: O' through the merge and the up-projection from given float32
partials, and the whole call's errors against those of its two roundings to bf16's eight bits."""

import numpy as np
import pytest
import torch

from oracle import view_oracle as V
from test_gpu_view import HEADS, Problem, clean_status, f64  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tokens,splits", [(1, 1), (20, 1), (32, 1), (33, 1), (200, 1), (1, 2), (32, 2), (33, 2), (130, 2),
                                           (40, 3), (5, 8), (60, 8), (9, 9), (40, 9), (3, 33), (2, 64)])
def test_the_finish_keeps_sixteen_bits(tokens, splits):
    """O' = 1 + d with |d| < 2^-9, whose first bf16 part is 1 in every column, over weights that cancel in pairs: the
    output is sum(d W) and comes from the second part alone.

    That part is d to eight bits: 2^-8 sum(|d| |W|) at the worst.  The products with the first part, 512 of at most |W|,
    are summed in float32 with steps of 2^-23 (truncated at the worst) of partial sums below max |W| (they cancel in
    neighbours): 512 x 2^-23 max |W|.  A merged value is off by S + 4 steps of 2^-24, the weights' common error cancels
    like the ones: (S + 4) 2^-24 sum |W|.  The result's rounding adds 2^-8 of it."""
    from mla_absorbed_decode_absorb_gb300 import ops
    g = torch.Generator().manual_seed(tokens * 100 + splits)
    max_kv = 64 * splits
    assert ops.mla_masked_num_splits(tokens, 1, max_kv, 1) == splits
    half = torch.randn(128, 128, 256, generator=g) * 0.02
    w = torch.stack([half, -half], -1).reshape(128, 128, 512).to(torch.bfloat16)
    d = (torch.rand(tokens, splits, 128, 512, generator=g) * 2 - 1) * 2.0 ** -9 * 0.99
    rows = 1.0 + d
    part_lse = torch.randn(tokens, splits, 128, generator=g)
    if splits > 2:
        part_lse[:, 1], rows[:, 1] = float("-inf"), 0.0  # a split without visible tokens
    ws = ops.alloc_masked_workspace(tokens, 1, max_kv, 1, device="cuda")
    latent = torch.full((tokens, 1, 128, 512), float("nan"), device="cuda")
    if splits == 1:
        latent[:, 0] = rows[:, 0].cuda()
    else:
        o_bytes = (rows.numel() * 4 + 255) // 256 * 256
        ws[:rows.numel() * 4] = rows.cuda().view(torch.uint8).flatten()
        ws[o_bytes:o_bytes + part_lse.numel() * 4] = part_lse.contiguous().cuda().view(torch.uint8).flatten()
    lse = torch.full((tokens, 1, 128), float("nan"), device="cuda")
    out = ops.mla_masked_combine_out_absorb(tokens, 1, max_kv, 1, ws, latent, w.cuda(), None, lse)
    share = torch.softmax(part_lse.double(), 1)
    total = (share[..., None] * (rows.double() - 1.0)).sum(1) if splits <= 2 else \
        (share[..., None] * torch.where(rows == 0, torch.zeros(()), rows.double() - 1.0)).sum(1)
    ref = torch.einsum("thm,hdm->thd", total, w.double())
    most = torch.einsum("thm,hdm->thd", total.abs(), w.double().abs())
    wsum = w.double().abs().sum(-1)[None]
    bound = 2.0 ** -8 * (ref.abs() + most) + 512 * 2.0 ** -23 * w.abs().max().item() + (splits + 4) * 2.0 ** -24 * wsum
    err = (out[:, 0].double().cpu() - ref).abs()
    assert (err <= bound).all(), (err / bound).max()
    assert bound.max() < 0.5 * ref.abs().max()  # the second part is seen
    if splits > 1:
        assert (lse[:, 0].double().cpu() - torch.logsumexp(part_lse.double(), 1)).abs().max() < 1e-5


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("split", [0, 1 << 20, 2])
def test_errors_are_those_of_two_roundings(fp8, split):
    """P has eight bits, and the output: uniform within half a step of 2^-8 at the worst, 2^-8 / sqrt(3) = 2.26e-3 rms of
    each.  Over zero-mean rows O' is off by the first of them, the output by both, sqrt(2) x 2.26e-3 = 3.2e-3; the second
    part of O' and float32 sums add less than 2^-14 of it."""
    prior, n_q = [1000, 333, 64], 6
    p = Problem(prior, n_q, seed=21, fp8=fp8)
    seen = [V.visible(L, n_q) for L in prior]
    out, lse, latent = p.run(split)
    w = f64(p.w_uv)[HEADS]
    e = np.zeros(4)
    for b in range(p.B):
        o_ref, _ = V.attend(f64(p.q[b])[:, HEADS], p.rows[b], seen[b])
        ref = np.einsum("nhm,hdm->nhd", o_ref, w)
        e += [((f64(out[b])[:, HEADS] - ref) ** 2).sum(), (ref ** 2).sum(),
              ((f64(latent[b])[:, HEADS] - o_ref) ** 2).sum(), (o_ref ** 2).sum()]
    assert (e[0] / e[1]) ** 0.5 < 3.2e-3 + 2e-4, (e[0] / e[1]) ** 0.5
    if p.splits == 1:
        assert (e[2] / e[3]) ** 0.5 < 2.26e-3 + 2e-4, (e[2] / e[3]) ** 0.5


@pytest.mark.parametrize("split", [2, 4])
def test_a_workspace_of_the_stated_size_is_enough(split):
    """Bytes on either side of it stay as they were, and one less is refused by both calls."""
    from mla_absorbed_decode_absorb_gb300 import ops
    B, n_q, max_kv = 3, 5, 700
    p = Problem([695, 100, 0], n_q, seed=5)
    n = ops.mla_masked_workspace_size(B, n_q, max_kv, split)
    room = torch.full((n + 512,), 0xA5, dtype=torch.uint8, device="cuda")
    ws = room[256:256 + n]
    q, cache, table, kv, w = (t.cuda() for t in (p.q, p.parts[0], p.table, p.kv(), p.w_uv))
    latent, lse = torch.empty(B, n_q, 128, 512, device="cuda"), torch.empty(B, n_q, 128, device="cuda")

    def attend(ws):
        ops.mla_decode_attn_masked_partial(q, cache, table, kv, n_q, max_kv, split, ws, latent, lse)

    def finish(ws):
        return ops.mla_masked_combine_out_absorb(B, n_q, max_kv, split, ws, latent, w, None, lse)
    attend(ws)
    out = finish(ws)
    assert (room[:256] == 0xA5).all() and (room[256 + n:] == 0xA5).all()
    want = p.run(split, max_kv=max_kv)
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    for call in (attend, finish):
        with pytest.raises(ops.MLAError):
            call(ws[:-1])
