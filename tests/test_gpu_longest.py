"""Calls whose bound on the lengths is the largest that 32 bits hold: the results of a tight bound, and a length that no
page table holds is reported."""

import pytest
import torch

from oracle import view_oracle as V
from test_gpu_view import HEADS, MLA_ERR_BOUNDS, Problem, clean_status  # noqa: F401

pytestmark = pytest.mark.gpu

LONGEST = 2 ** 31 - 1


def status():
    from mla_absorbed_decode_absorb_gb300 import ops
    torch.cuda.synchronize()
    return ops.mla_get_device_status()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("window,sinks,split", [(0, 0, 0), (0, 0, LONGEST), (0, 0, 1 << 24), (100, 4, 0), (100, 4, 1),
                                                (LONGEST, LONGEST, 0)])
def test_masked_attention(fp8, window, sinks, split):
    prior, n_q = [0, 63, 500], 3
    p = Problem(prior, n_q, seed=window % 97 + split % 89, fp8=fp8)
    seen = [V.visible(L, n_q, window, sinks) for L in prior]
    for bound in (LONGEST, LONGEST - 62, LONGEST - 63):
        result = p.run(split, window, sinks, max_kv=bound)
        p.check(result, seen, HEADS)
    for long in (LONGEST, LONGEST - 63):
        p.kv = lambda long=long: torch.tensor([3, long, 503], dtype=torch.int32)
        out, lse, _ = p.run(split, window, sinks, max_kv=LONGEST)
        assert status() == MLA_ERR_BOUNDS
        assert not out[1].any() and torch.isneginf(lse[1]).all()
        assert torch.equal(out[::2], result[0][::2]) and torch.equal(lse[::2], result[1][::2])


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("split", [0, LONGEST, 1 << 25, 1 << 24, 1 << 23])
def test_causal_attention(fp8, split):
    """The same pages a split, so the same results, as with the bound of the longest sequence; where the plan chooses, to
    both calls' roundings."""
    from mla_absorbed_decode_absorb_gb300 import ops
    prior, n_q = [0, 63, 5000], 3
    p = Problem(prior, n_q, seed=3, fp8=fp8)
    q, table, kv, w = (t.cuda() for t in (p.q, p.table, p.kv(), p.w_uv))
    cache = tuple(x.cuda() for x in p.parts)
    attend = ops.mla_decode_attn_fp8_partial if fp8 else ops.mla_decode_attn_partial

    def run(max_kv, split, kv=kv):
        ws = ops.alloc_workspace(3, n_q, max_kv, split, "cuda")
        latent, lse = torch.empty(3, n_q, 128, 512, device="cuda"), torch.empty(3, n_q, 128, device="cuda")
        attend(q, cache if fp8 else cache[0], table, kv, n_q, max_kv, split, ws, latent, lse)
        return ops.mla_combine_out_absorb(3, n_q, max_kv, split, ws, latent, w, None, lse), lse
    want = run(5003, 1 << 20)
    for bound in (LONGEST, LONGEST - 62, LONGEST - 63):
        out, lse = run(bound, split)
        # splits that hold no token leave the first one's partial, in bf16 where there are several (half a step, 2^-8)
        tol = 2.0 ** -6 if split in (0, 1 << 24, 1 << 23) else 0.0
        assert (out.float() - want[0].float()).abs().max() <= tol * want[0].float().abs().max()
        assert (lse - want[1]).abs().max() <= (5e-3 if split == 0 else 1e-5 if tol else 0.0)
    for long in (LONGEST, LONGEST - 63):
        out, lse = run(LONGEST, split, torch.tensor([3, long, 5003], dtype=torch.int32, device="cuda"))
        assert status() == MLA_ERR_BOUNDS
        assert not out[1].any() and torch.isneginf(lse[1]).all()


@pytest.mark.parametrize("past", [1, 70])
def test_prompts_behind_a_context_that_wraps(past):
    """seq_lens_before so large that n_q more pass 32 bits, and kv_lens the sum that has: reported, and zeros."""
    from mla_absorbed_decode_absorb_gb300 import ops
    from test_gpu_view import prompt
    n_q = 70
    out, lse, (q, r, lens, rope, cache, table, kv, uk, uv, max_kv) = prompt([100, 100], n_q, 50, 4, 6, poison=False)
    k, v = ops.mla_decompress_kv(cache, table, kv, max_kv, uk, uv)
    lens, kv = lens.clone(), kv.clone()
    lens[1], kv[1] = 2 ** 31 - past, n_q - past - 2 ** 31
    for call, args in ((ops.mla_prefill_attn, ()), (ops.mla_prefill_attn_window, (50, 4))):
        got_lse = torch.empty_like(lse)
        got = call(q, r, lens, rope, k, v, cache, table, kv, *args, None, got_lse)
        assert status() == MLA_ERR_BOUNDS
        assert not got[1].any() and torch.isneginf(got_lse[1]).all() and torch.isfinite(got_lse[0]).all()
