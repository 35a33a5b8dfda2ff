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
