"""The few-bit operators in the calls that a program may make of them: values at the ends of bf16's range, both
projections of a pair the same, first calls from two threads, graphs side by side, and the sessions' further paths."""

import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from oracle import few_bits_oracle as F
from test_gpu_few_bits import check_norm, f64, linear_inputs, linear_ref, norm_inputs, ok, run_linear, within
from test_gpu_streams import same_bits

pytestmark = pytest.mark.gpu

SHAPES = [(1, 320, 70), (8, 1024, 40), (9, 1088, 16601), (40, 320, 24000), (64, 320, 14500), (100, 1088, 2600),
          (256, 4160, 3000)]


@pytest.mark.parametrize("T,K,N", SHAPES)
@pytest.mark.parametrize("xe,we", [(-131, 100), (-131, 120), (-126, 0), (110, -100)])
def test_linear_of_small_and_large_values(T, K, N, xe, we):
    """bf16 x below and at the top of its normal range with scales the other way: a value is not lost before it is
    scaled.  An x of 2^-131 has three bits; the products are exact all the same.  fp32 sums below 2^-126 are rounded to
    multiples of 2^-149, half of one each in K products and three operations of a group, times the scale; y below
    2^-126 to multiples of 2^-133."""
    x, _, w4, scale = linear_inputs(T, K, N, False, T + K)
    x = (x.double() * 2.0 ** xe).to(torch.bfloat16)
    scale = (scale.double() * 2.0 ** we).to(torch.bfloat16)
    assert torch.isfinite(x.float()).all() and torch.isfinite(scale.float()).all()
    ref, tol = linear_ref(x, None, w4, scale)
    tol = tol + 2.0 ** -134 + (K + 3 * F.groups(K)) * 2.0 ** -150 * max(1.0, float(f64(scale).max()))
    assert 0 < np.abs(ref).max() < 2.0 ** 120
    y = run_linear(x, None, w4, scale)
    within(f64(y), ref, tol)
    if xe == -131:
        assert (f64(y) != 0).mean() > 0.9  # the smallest values count
    ok()


@pytest.mark.parametrize("T,K,N", SHAPES)
@pytest.mark.parametrize("fp8", [False, True])
def test_a_pair_of_one_weight(T, K, N, fp8):
    from mla_absorbed_decode_absorb_gb300 import ops
    x, sx, w4, scale = (t if t is None else t.cuda() for t in linear_inputs(T, K, N, fp8, T))
    w = (w4, scale)
    y0, y1 = ops.mla_linear_w4_fp8_pair(x, sx, w, w) if fp8 else ops.mla_linear_w4_pair(x, w, w)
    assert y0.data_ptr() != y1.data_ptr() and same_bits(y0, y1)
    ref, tol = linear_ref(*linear_inputs(T, K, N, fp8, T))
    within(f64(y0), ref, tol)
    ok()


def test_norm_in_place_with_both_outputs():
    """x, the residual and the bf16 output in place, with the 8-bit output beside them."""
    from mla_absorbed_decode_absorb_gb300 import ops
    for T, D in ((3, 7168), (2000, 512), (400, 7168), (3, 16384)):
        x, r, w = norm_inputs(T, D, 91)
        x = x.contiguous()
        x0, r0 = x.clone(), r.clone()
        y8, s = ops.mla_rms_norm_fp8(x, w, 1e-6, r, y=x)
        check_norm(x0, r0, w, 1e-6, r_out=r, y=x, y8=y8, scale=s)
    ok()


def test_first_calls_from_two_threads():
    """A process whose first calls of every kernel come from two threads at once, on streams of their own."""
    code = """
import threading
import torch
from mla_absorbed_decode_absorb_gb300 import ops
g = torch.Generator(device="cuda").manual_seed(0)
w = torch.randn(9000, 4160, generator=g, device="cuda").to(torch.bfloat16)
xs = [torch.randn(t, 4160, generator=g, device="cuda").to(torch.bfloat16) for t in (1, 16, 40, 64, 200)]
gamma = torch.ones(4160, dtype=torch.bfloat16, device="cuda")
torch.cuda.synchronize()
out, gate = [None, None], threading.Barrier(2)

def calls(i):
    with torch.cuda.stream(torch.cuda.Stream()):
        gate.wait()
        w4, s = ops.mla_quantize_w4(w)
        got = [ops.mla_dequantize_w4(w4, s)]
        for x in xs:
            y8, ys = ops.mla_rms_norm_fp8(x, gamma)
            got += [ops.mla_linear_w4(x, w4, s), ops.mla_linear_w4_fp8(y8, ys, w4, s)]
        torch.cuda.current_stream().synchronize()
        out[i] = got

threads = [threading.Thread(target=calls, args=(i,)) for i in range(2)]
[t.start() for t in threads]
[t.join() for t in threads]
assert len(out[0]) == len(out[1]) == 11
assert all(torch.equal(a.view(torch.int16), b.view(torch.int16)) for a, b in zip(*out))
assert ops.mla_get_device_status() == ops.MLA_OK
print("both")
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "both" in r.stdout, r.stderr[-2000:]


def test_two_graphs_side_by_side():
    """Two captured projections replayed on two streams at once, and their eager calls between: no workspace is shared."""
    from mla_absorbed_decode_absorb_gb300 import ops
    graphs = []
    for T, K, N in ((5, 7168, 577), (200, 7168, 1536)):
        x, _, w4, scale = (t if t is None else t.cuda() for t in linear_inputs(T, K, N, False, T))
        ref = ops.mla_linear_w4(x, w4, scale)
        y, stream = torch.empty_like(ref), torch.cuda.Stream()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            for _ in range(20):
                ops.mla_linear_w4(x, w4, scale, y)
        graphs.append((graph, stream, y, ref, (x, w4, scale)))
    for graph, stream, y, _, _ in graphs:
        y.zero_()
    torch.cuda.synchronize()
    again = []
    for _ in range(5):
        for graph, stream, _, _, args in graphs:
            with torch.cuda.stream(stream):
                graph.replay()
            again.append(ops.mla_linear_w4(*args))
    torch.cuda.synchronize()
    for i, (_, _, y, ref, _) in enumerate(graphs):
        assert same_bits(y, ref) and all(same_bits(z, ref) for z in again[i::2])
    ok()


@pytest.mark.parametrize("kw", [{}, dict(overlap_append=True)])
def test_prefill_over_the_fp8_cache_captured(kw):
    """The non-absorbed path over an FP8 cache as one graph, and with the append on a stream of its own: the bits of the
    plain step."""
    from mla_absorbed_decode_absorb_gb300 import runtime
    from mla_absorbed_decode_absorb_gb300 import workloads as W
    inp = W.generate(W.custom("captured", [0, 63, 130, 300], n_q=70, cache_format="fp8"), seed=33)
    s = runtime.DecodeSession(inp)
    s.step()
    torch.cuda.synchronize()
    t = runtime.DecodeSession(inp, **kw)
    graph = t.capture() if hasattr(t, "capture") else runtime.StepGraph(t)
    for _ in range(2):
        t.out.zero_(), t.lse.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert same_bits(t.out, s.out) and same_bits(t.lse, s.lse)
    t.out.zero_()
    t.step()
    torch.cuda.synchronize()
    assert same_bits(t.out, s.out)
    ok()
