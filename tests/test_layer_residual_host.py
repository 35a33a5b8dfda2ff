"""Which residuals a layer session takes, without a GPU (every refusal comes before the session is laid out)."""

import contextlib

import pytest
import torch

from mla_absorbed_decode_absorb_gb300 import workloads as W


class LaidOut(Exception):
    pass


@pytest.fixture
def session(monkeypatch):
    """session(residual) -> "taken" once the arguments have been accepted."""
    from mla_absorbed_decode_absorb_gb300.runtime import LayerNorms, LayerSession
    li = W.generate_layer(W.Workload("residual", batch=2, n_q=2, lengths=(0, 5), d_model=256), seed=3)
    ones = [torch.ones(n, dtype=torch.bfloat16) for n in (256, W.D_Q_LATENT, W.D_LATENT)]

    def stop(*a, **k):
        raise LaidOut
    monkeypatch.setattr(LayerSession, "_lay_out", stop)
    monkeypatch.setattr("mla_absorbed_decode_absorb_gb300.runtime._laid_out_on", lambda *a: contextlib.nullcontext())

    def build(residual, device="cpu"):
        try:
            LayerSession(li, device=device, norms=LayerNorms(*ones), residual=residual)
        except LaidOut:
            return "taken"
    return build


def z(*shape, dtype=torch.bfloat16, device=None):
    return torch.zeros(*shape, dtype=dtype, device=device)


def test_residuals_that_are_taken(session):
    assert session(z(2, 2, 256)) == session(z(4, 256)) == "taken"
    # a host tensor is copied to the device, dense or not
    assert session(z(256, 4).t(), device="meta") == "taken"


def test_residuals_that_are_refused(session):
    """A tensor of the session's own device is added to in place: one that would have to be copied for that is refused
    rather than left behind."""
    for bad in (z(256, 4).t(), z(4, 512)[:, ::2], z(4, 512)[:, :256]):
        with pytest.raises(ValueError, match="in place"):
            session(bad)
    for bad in (z(2, 256), z(5, 256), z(1)):
        with pytest.raises(ValueError, match="elements"):
            session(bad)
    with pytest.raises(TypeError):
        session(z(4, 256, dtype=torch.float32))
    with pytest.raises(ValueError, match="device"):
        session(z(4, 256, device="meta"))  # neither the host's nor the session's
