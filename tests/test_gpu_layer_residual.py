"""The residual stream of a layer session: whose memory it is, and what a capture leaves of it."""

import pytest
import torch

from mla_absorbed_decode_absorb_gb300 import workloads as W
from test_gpu_layer import SMALL
from test_gpu_layer_few_bits import norms
from test_gpu_streams import same_bits

pytestmark = pytest.mark.gpu


def residual_of(li, seed=4):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(li.x.shape, generator=g).to(torch.bfloat16)


@pytest.mark.parametrize("kw", [{}, dict(weights="w4", activations="fp8")])
def test_a_capture_leaves_the_residual_as_it_was(kw):
    """The warm-up steps in front of a capture add to the residual: it is put back.  Replays then do what steps do."""
    from mla_absorbed_decode_absorb_gb300 import ops
    from mla_absorbed_decode_absorb_gb300.runtime import LayerSession, StepGraph
    li = W.generate_layer(SMALL["mtp"], seed=21)
    n, r = norms(li, 2), residual_of(li)
    s = LayerSession(li, norms=n, residual=r, **kw)
    eager = []
    for _ in range(3):
        s.step()
        torch.cuda.synchronize()
        eager.append((s.residual.clone(), s.y.clone()))
    for capture in (lambda t: t.capture(), lambda t: t.capture(warmup=1), StepGraph):
        t = LayerSession(li, norms=n, residual=r, **kw)
        graph = capture(t)
        torch.cuda.synchronize()
        assert same_bits(t.residual.cpu().reshape(r.shape), r)
        for res, y in eager:
            graph.replay()
            torch.cuda.synchronize()
            assert same_bits(t.residual, res) and same_bits(t.y, y)
    assert ops.mla_get_device_status() == ops.MLA_OK


def test_whose_memory_the_residual_is():
    """A tensor of the device is added to in place and may be shared by layers; a host tensor, dense or not, is copied
    and stays as it is."""
    from mla_absorbed_decode_absorb_gb300.runtime import LayerSession
    li = W.generate_layer(SMALL["mtp"], seed=22)
    n, r = norms(li, 3), residual_of(li)
    shared = r.cuda()
    layers = [LayerSession(li, norms=n, residual=shared) for _ in range(2)]
    assert all(s.residual.data_ptr() == shared.data_ptr() for s in layers)
    strided = r.reshape(-1, li.workload.d_model).t().contiguous().t()
    assert not strided.is_contiguous()
    for host in (r, strided):
        before = host.clone()
        own = LayerSession(li, norms=n, residual=host)
        own.step()
        torch.cuda.synchronize()
        once = (li.x.float() + r.float()).to(torch.bfloat16).cuda()
        assert same_bits(own.residual.view(once.shape), once) and torch.equal(host.float(), before.float())
    for s in layers:
        s.step()
    own.step()
    torch.cuda.synchronize()
    assert same_bits(shared.view(own.residual.shape), own.residual)
