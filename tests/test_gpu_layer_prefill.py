"""The decode layer with 64 or more new tokens a sequence: its projections and norms around the non-absorbed path,
over the bf16 and the FP8 cache, in every weight and activation format.

bf16 cache: the tolerance of the layer with few tokens, from the same roundings.  FP8 cache: the definition continues
from the cache's dequantised rows, read back by the operator whose bits are tested elsewhere; same tolerance."""

import numpy as np
import pytest
import torch

from oracle import mla_oracle as O
from mla_absorbed_decode_absorb_gb300 import workloads as W
from test_gpu_few_bits import f64
from test_gpu_layer import Y_REL_L2
from test_gpu_layer_few_bits import check, norms, run, weight
from test_gpu_parity import rel_l2
from test_gpu_streams import same_bits

pytestmark = pytest.mark.gpu

FORMS = [dict(), dict(weights="w4"), dict(norm=True, weights="w4", activations="fp8", res=True)]


def layer(cache_format, form, seed):
    wl = W.Workload("layer_chunk", batch=2, n_q=70, lengths=(0, 130), d_model=1024, cache_format=cache_format)
    li, kw, residual = W.generate_layer(wl, seed=seed), dict(form), None
    if kw.pop("norm", False):
        kw["norms"] = norms(li, 3)
    if kw.pop("res", False):
        residual = torch.randn(li.x.shape, generator=torch.Generator().manual_seed(4)).to(torch.bfloat16)
        kw["residual"] = residual.clone()
    s = run(li, **kw)
    assert s.dec.path == "non_absorbed" and s.T == 140
    return li, s, residual


@pytest.mark.parametrize("form", FORMS)
def test_layer_of_a_chunk(form):
    li, s, residual = layer("bf16", form, 41)
    check(s, li, residual)


@pytest.mark.parametrize("form", FORMS)
def test_layer_of_a_chunk_over_the_fp8_cache(form):
    """From the per-head output on the layer is its projection; the attention's own output is that of a decode session
    over the same rows, taken apart in the prefill tests."""
    li, s, _ = layer("fp8", form, 42)
    assert "read_back" in s.stage_names()
    out = f64(s.dec.out).reshape(s.T, -1)
    y = O.linear(out, weight(s, li, "w_o"))
    assert rel_l2(f64(s.y), y) <= Y_REL_L2
    # the same step with the cache's rows in a bf16 cache: the attention reads what the read back wrote
    from mla_absorbed_decode_absorb_gb300 import ops
    d = s.dec
    rows = ops.mla_read_kv_fp8(d.cache_fp8, d.page_table, d.kv_lens, d.max_kv_len)
    assert same_bits(rows, d.kv_rows)
    k, v = ops.mla_decompress_kv(rows, d.kv_table, d.kv_lens, d.max_kv_len, d.w_uk, d.w_uv)
    again = ops.mla_prefill_attn(d.q_nope, d.q_rope, d.prior_lens, d.rope, k, v, rows, d.kv_table, d.kv_lens)
    torch.cuda.synchronize()
    assert same_bits(again, d.out) and np.isfinite(out).all() and np.abs(out).max() > 0
    # replayed, it gives the same bits (the residual is part of the step's state)
    before = None if s.residual is None else s.residual.clone()
    graph = s.capture()
    if before is not None:
        assert same_bits(s.residual, before)
    first = None
    for _ in range(2):
        if before is not None:
            s.residual.copy_(before)
        graph.replay()
        torch.cuda.synchronize()
        assert first is None or same_bits(s.y, first)
        first = s.y.clone()
    assert ops.mla_get_device_status() == ops.MLA_OK
