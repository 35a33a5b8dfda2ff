"""Calls on a stream of the caller's while the current stream is busy: what a call makes itself must not wait there."""

import numpy as np
import pytest
import torch

from test_gpu_few_bits import fp8_cache, ok, to_gpu

pytestmark = pytest.mark.gpu

BUSY = 400_000_000  # clock cycles, about 0.2 s


def same_bits(a, b):
    return torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_read_back_on_another_stream_while_the_current_one_is_busy():
    """The rows that the call makes are filled with the sentinel before they are read into, wherever it runs."""
    from mla_absorbed_decode_absorb_gb300 import ops
    c8, scale, kr, pt, lens = fp8_cache([3000, 64, 0, 1], 71)
    cache, ptg, ng = to_gpu(c8, scale, kr, pt, lens)
    ref = ops.mla_read_kv_fp8(cache, ptg, ng, 3000)
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        torch.cuda.synchronize()
        torch.cuda._sleep(BUSY)
        rows = ops.mla_read_kv_fp8(cache, ptg, ng, 3000, stream=stream)
        side.synchronize()
        first = rows.to("cpu", non_blocking=False)
        torch.cuda.synchronize()
        assert same_bits(rows, ref) and same_bits(first, ref.cpu())
    assert np.isnan(ref.view(4, -1)[2].float().cpu().numpy()).all()
    ok()
