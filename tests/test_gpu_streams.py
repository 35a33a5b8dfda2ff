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


@pytest.mark.parametrize("n_q,cache_format", [(70, "fp8"), (70, "bf16"), (2, "bf16"), (2, "fp8")])
def test_a_session_laid_out_on_a_busy_stream(n_q, cache_format, monkeypatch):
    """A session whose constructor's stream has work in front of it and between the pools' fills, stepped on yet
    another stream at once: the bits of a session of the current stream.  Sequences of one length, whose histories
    are copied into the same memory one after the other."""
    from mla_absorbed_decode_absorb_gb300 import runtime
    from mla_absorbed_decode_absorb_gb300 import workloads as W
    inp = W.generate(W.custom("busy", [130, 130, 130, 0], n_q=n_q, cache_format=cache_format), seed=8)
    s = runtime.DecodeSession(inp)
    s.step()
    torch.cuda.synchronize()
    real = runtime.empty_cache

    def slow_empty_cache(*args):
        torch.cuda._sleep(BUSY)
        return real(*args)

    monkeypatch.setattr(runtime, "empty_cache", slow_empty_cache)
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    with torch.cuda.stream(a):
        torch.cuda._sleep(BUSY)
    t = runtime.DecodeSession(inp, stream=a)
    t.step(b)
    b.synchronize()
    assert same_bits(t.out, s.out) and same_bits(t.lse, s.lse)
    ok()


@pytest.mark.parametrize("kind", ["fold", "few_bits"])
def test_a_layer_laid_out_on_a_busy_stream(kind):
    """Folded and quantised weights, whose inputs are given back while the constructor's stream is still busy."""
    from mla_absorbed_decode_absorb_gb300 import runtime
    from mla_absorbed_decode_absorb_gb300 import workloads as W
    li = W.generate_layer(W.Workload("busy", batch=2, n_q=2, lengths=(5, 130), d_model=1024), seed=9)
    kw = {"fold": dict(fold=True), "few_bits": dict(weights="w4")}[kind]
    s = runtime.LayerSession(li, **kw)
    s.step()
    torch.cuda.synchronize()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    with torch.cuda.stream(a):
        torch.cuda._sleep(BUSY)
    t = runtime.LayerSession(li, stream=a, **kw)
    t.step(b)
    b.synchronize()
    assert same_bits(t.y, s.y)
    ok()


def test_outputs_of_another_stream_share_no_memory_with_pending_work():
    """An output made on a side stream: not in memory whose last use on the current stream is still to come, neither
    what the current stream gave back before the call nor an earlier output that it still reads."""
    from mla_absorbed_decode_absorb_gb300 import ops
    g = torch.Generator(device="cuda").manual_seed(3)
    T, K, N = 8, 1024, 4096
    w4, scale = ops.mla_quantize_w4(torch.randn(N, K, generator=g, device="cuda").to(torch.bfloat16))
    x1, x2 = (torch.randn(T, K, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    ref1, ref2 = ops.mla_linear_w4(x1, w4, scale), ops.mla_linear_w4(x2, w4, scale)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(2):
        scratch = torch.empty_like(ref1)
        torch.cuda._sleep(BUSY)
        scratch.fill_(7.0)
        del scratch  # given back, but written later
        y = ops.mla_linear_w4(x1, w4, scale, stream=side)
        side.synchronize()
        torch.cuda.synchronize()
        assert same_bits(y, ref1)
        torch.cuda._sleep(BUSY)
        later = y.clone()
        del y  # given back, but read later
        y = ops.mla_linear_w4(x2, w4, scale, stream=side)
        torch.cuda.synchronize()
        assert same_bits(later, ref1) and same_bits(y, ref2)
        del y, later
    ok()
