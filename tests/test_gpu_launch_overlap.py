"""The 4-bit projections behind a kernel that runs for longer than a bounded wait."""

import numpy as np
import pytest
import torch

from test_gpu_few_bits import f64, linear_inputs, linear_ref, ok, within

pytestmark = pytest.mark.gpu


def long_attention(pages):
    """The decode attention of one sequence, unsplit, over one page again and again: two CTAs that release the next
    kernel at their start and stream `pages` pages."""
    from mla_absorbed_decode_absorb_gb300 import ops
    q = torch.zeros(1, 1, 128, 576, dtype=torch.bfloat16, device="cuda")
    cache = torch.zeros(1, 64, 576, dtype=torch.bfloat16, device="cuda")
    table = torch.zeros(1, pages, dtype=torch.int32, device="cuda")
    lens = torch.full((1,), 64 * pages, dtype=torch.int32, device="cuda")
    o = torch.empty(1, 1, 128, 512, dtype=torch.float32, device="cuda")
    args = (q, cache, table, lens, 1, 64 * pages, pages, None, o)
    assert ops.mla_decode_num_splits(1, 1, 64 * pages, pages) == 1
    return lambda: ops.mla_decode_attn_partial(*args)


def seconds(call):
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    call()
    end.record()
    torch.cuda.synchronize()
    return start.elapsed_time(end) / 1e3


def test_projections_behind_a_long_kernel():
    """At launch overlap 2 a projection starts while the kernel before it runs.  Its waits of at most 2 s begin when that
    one has finished: nothing is given up, whichever kernel and tile."""
    from mla_absorbed_decode_absorb_gb300 import ops
    before = ops.mla_get_launch_overlap()
    some = 100_000
    long_attention(1000)()
    per_page = seconds(long_attention(some)) / some
    pages = int(2.6 / per_page)
    assert 64 * pages < 2 ** 31
    behind = long_attention(pages)
    cases = [(T, K, N, fp8) for T, K, N in ((3, 512, 64), (16, 7168, 2561), (64, 1536, 3001), (100, 1088, 2600),
                                            (256, 4160, 3000)) for fp8 in (False, True)]
    ops.mla_set_launch_overlap(2)
    try:
        for T, K, N, fp8 in cases:
            x, sx, w4, scale = (t if t is None else t.cuda() for t in linear_inputs(T, K, N, fp8, T))
            y = torch.zeros(T, N, dtype=torch.bfloat16, device="cuda")
            torch.cuda.synchronize()

            def both():
                behind()
                if fp8:
                    ops.mla_linear_w4_fp8(x, sx, w4, scale, y)
                else:
                    ops.mla_linear_w4(x, w4, scale, y)
            assert seconds(both) > 2.2
            ok()
            ref, tol = linear_ref(*linear_inputs(T, K, N, fp8, T))
            within(f64(y), ref, tol)
            assert np.abs(ref).max() > 0.1
    finally:
        ops.mla_set_launch_overlap(before)
