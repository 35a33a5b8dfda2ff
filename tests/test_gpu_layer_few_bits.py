"""The decode layer with norms, 4-bit weights and 8-bit activations, and prefill over the FP8 cache.

The layer's roundings to bf16 against the float64 definition: the five of the
plain layer (c^Q, q^C, q^R, O, y) and up to four more (the normed hidden state, c^KV
before its norm, c^Q after, and the residual's sum does not count: the norm reads it
unrounded).  Each is at most 2^-8 of its value, 2^-8 / sqrt(3) in the mean square at
worst; nine of them and the attention's own 5e-3 add in quadrature to 8.4e-3: the
plain layer's tolerance of 1e-2 holds.  4-bit weights are taken as the values that
they stand for, so they add nothing; 8-bit activations likewise (the definition
continues from the codes the norm wrote, which are checked against the norm's own
definition).
"""

import numpy as np
import pytest
import torch

from oracle import few_bits_oracle as F
from oracle import mla_oracle as O
from mla_absorbed_decode_absorb_gb300 import workloads as W
from test_gpu_fp8 import oracle_fp8_images, oracle_sequence_fp8
from test_gpu_layer import SMALL, Y_REL_L2, f64
from test_gpu_parity import bits, rel_l2
from test_gpu_prefill import LSE_MAX_ABS, O_MAX_ABS, O_REL_L2

pytestmark = pytest.mark.gpu


def norms(li, seed):
    from mla_absorbed_decode_absorb_gb300.runtime import LayerNorms
    g = torch.Generator().manual_seed(seed)

    def w(n):
        return (1 + 0.2 * torch.randn(n, generator=g)).to(torch.bfloat16)
    return LayerNorms(w(li.workload.d_model), w(W.D_Q_LATENT), w(W.D_LATENT), 1e-5)


def run(li, **kw):
    from mla_absorbed_decode_absorb_gb300 import ops
    from mla_absorbed_decode_absorb_gb300.runtime import LayerSession
    s = LayerSession(li, **kw)
    s.step()
    torch.cuda.synchronize()
    assert ops.mla_get_device_status() == ops.MLA_OK
    return s


def weight(s, li, name):
    """The float64 weight [out, in] the session's projection uses."""
    w = getattr(s, name)
    if isinstance(w, tuple):
        return F.weights_w4(w[0].cpu().numpy(), f64(w[1]))
    return f64(w)


def normed(x, w, eps, got, residual=None):
    """The norm's output as the layer goes on with it: the definition's, or for 8 bits the codes' values, which have
    to be within half a step of it."""
    _, v = F.rms_norm(x, f64(w), eps, residual)
    if not isinstance(got, tuple):
        return v
    codes, scale = got[0].cpu().numpy(), got[1].double().cpu().numpy()
    value, step = F.activations_fp8(codes, scale), F.per_column(scale, v.shape[1])
    # c^Q is rounded to bf16 before its norm: 2^-8 of an element, and of the row's root mean square
    near = np.maximum(2.0 ** -4 * np.abs(v), 2.0 ** -10 * step) + 2 * 2.0 ** -8 * np.abs(v)
    assert (np.abs(value - v) <= near * (1 + 2.0 ** -7)).all()
    return value


def oracle(s, li, residual=None):
    """(y, O) of every sequence, from the definition."""
    inp, nq = li.base, li.workload.n_q
    n = s.norms
    x = f64(li.x).reshape(s.T, -1)
    r = None if residual is None else f64(residual).reshape(s.T, -1)
    if n is not None:
        x = normed(x, n.hidden, n.eps, s._x_normed, r)
    c_new = O.linear(x, weight(s, li, "w_dkv"))
    k_new = O.linear(x, weight(s, li, "w_kr"))
    c_q = O.linear(x, weight(s, li, "w_dq"))
    if n is not None:
        _, c_new = F.rms_norm(c_new, f64(n.kv_latent), n.eps)
        c_q = normed(c_q, n.q_latent, n.eps, s._cq_normed)
    q_nope = O.linear(c_q, weight(s, li, "w_uq")).reshape(s.T, 128, 128)
    q_rope = O.linear(c_q, weight(s, li, "w_qr")).reshape(s.T, 128, 64)
    ys, os_ = [], []
    for b in range(inp.batch):
        t = slice(b * nq, (b + 1) * nq)
        hc, hk = inp.history(b)
        L = int(inp.prior_lens[b])
        rows = O.bf16_bits_to_f64(O.f32_to_bf16_bits(c_new[t].astype(np.float32)))
        kr_new = O.bf16_bits_to_f64(O.rope_key_bf16_bits(O.f32_to_bf16_bits(k_new[t].astype(np.float32)),
                                                         L + np.arange(nq)))
        kr = O.bf16_bits_to_f64(O.rope_key_bf16_bits(bits(hk), np.arange(L))) if L else np.zeros((0, 64))
        c = np.concatenate([f64(hc) if L else np.zeros((0, 512)), rows])
        o, _, _ = O.decode_mha(q_nope[t], q_rope[t], f64(inp.w_uk), f64(inp.w_uv), c, np.concatenate([kr, kr_new]), L)
        os_.append(o)
        ys.append(O.linear(o.reshape(nq, -1), weight(s, li, "w_o")))
    return np.concatenate(ys), np.concatenate(os_)


def check(s, li, residual=None):
    y, o = oracle(s, li, residual)
    got = s.y.float().cpu().numpy()
    assert np.isfinite(got).all()
    assert rel_l2(s.dec.out.float().cpu().numpy().reshape(o.shape), o) <= Y_REL_L2
    assert rel_l2(got, y) <= Y_REL_L2, rel_l2(got, y)


@pytest.mark.parametrize("name", sorted(SMALL))
@pytest.mark.parametrize("kw", [dict(weights="w4"), dict(norm=True), dict(norm=True, weights="w4"),
                                dict(norm=True, weights="w4", activations="fp8"),
                                dict(norm=True, weights="w4", activations="fp8", res=True)])
def test_layer_few_bits(name, kw):
    li = W.generate_layer(SMALL[name], seed=15)
    kw = dict(kw)
    residual = None
    if kw.pop("norm", False):
        kw["norms"] = norms(li, 3)
    if kw.pop("res", False):
        g = torch.Generator().manual_seed(4)
        residual = torch.randn(li.x.shape, generator=g).to(torch.bfloat16)
        kw["residual"] = residual.clone()
    s = run(li, **kw)
    check(s, li, residual)
    if residual is not None:
        h = f64(li.x) + f64(residual)
        got = f64(s.residual).reshape(h.shape)
        assert (np.abs(got - h) <= (2.0 ** -8 + 2.0 ** -24) * np.abs(h)).all()
    assert s.stage_names()[0] == ("norm_in" if "norms" in kw else "proj_kv")


def test_layer_folds_take_the_norms():
    """The weight pre-folds behind the normed c^Q: one more rounding of the folded weights, the same tolerance (as
    without norms)."""
    li = W.generate_layer(SMALL["mtp"], seed=16)
    s = run(li, norms=norms(li, 5), fold=True)
    y, _ = oracle(s, li)
    assert rel_l2(s.y.float().cpu().numpy(), y) <= Y_REL_L2


def test_layer_few_bits_captured():
    """The whole step as one graph, replayed on another hidden state: the bits of the same session called eagerly."""
    li = W.generate_layer(SMALL["edges"], seed=17)
    kw = dict(norms=norms(li, 6), weights="w4", activations="fp8")
    s = run(li, **kw)
    first = s.y.clone()
    graph = s.capture()
    g = torch.Generator().manual_seed(7)
    x2 = torch.randn(s.x.shape, generator=g).to(torch.bfloat16).cuda()
    x1 = s.x.clone()
    out = []
    for x in (x1, x2, x1):
        s.x.copy_(x)
        graph.graph.replay()
        torch.cuda.synchronize()
        out.append(s.y.clone())
    s.x.copy_(x2)
    s.step()
    torch.cuda.synchronize()
    assert torch.equal(out[0].view(torch.int16), first.view(torch.int16))
    assert torch.equal(out[2].view(torch.int16), first.view(torch.int16))
    assert torch.equal(out[1].view(torch.int16), s.y.view(torch.int16))


def test_layer_counts_its_launches():
    from mla_absorbed_decode_absorb_gb300 import ops
    li = W.generate_layer(SMALL["edges"], seed=18)
    plain = run(li)
    assert run(li, norms=norms(li, 1)).launches_per_step() == plain.launches_per_step() + 3
    few = run(li, weights="w4")
    # six projections in four launches
    assert few.launches_per_step() == few.dec.launches_per_step() + 4
    assert ops.mla_get_device_status() == ops.MLA_OK


def test_layer_refusals():
    from mla_absorbed_decode_absorb_gb300.runtime import LayerSession
    li = W.generate_layer(SMALL["mtp"], seed=1)
    n = norms(li, 1)
    for kw in [dict(weights="w3"), dict(activations="int8"), dict(weights="w4", fold=True),
               dict(activations="fp8"), dict(activations="fp8", weights="w4"), dict(activations="fp8", norms=n),
               dict(residual=li.x)]:
        with pytest.raises(ValueError):
            LayerSession(li, **kw)


def test_prefill_over_the_fp8_cache():
    """A chunk of 64 or more new tokens over an FP8 cache: append, read back, decompress, attention, against the
    definition on the dequantised values.  The rows read back are rounded to bf16 (2^-8 at most on keys and values,
    about 1.1e-3 in the mean square), which in quadrature leaves the prefill path's tolerances as they are."""
    from mla_absorbed_decode_absorb_gb300 import ops
    from mla_absorbed_decode_absorb_gb300.runtime import DecodeSession
    inp = W.generate(W.custom("prefill_fp8", [0, 63, 130, 300], n_q=70, cache_format="fp8"), seed=31)
    s = DecodeSession(inp)
    assert s.path == "non_absorbed" and s.stage_names() == ["append", "read_back", "decompress", "prefill_attn"]
    assert s.launches_per_step() == 4
    s.step()
    torch.cuda.synchronize()
    assert ops.mla_get_device_status() == ops.MLA_OK
    heads = [0, 41, 127]
    img = oracle_fp8_images(inp)
    got, lse = s.out.float().cpu().numpy(), s.lse.cpu().numpy()
    o_all, r_all = [], []
    for b in range(inp.batch):
        o_ref, _, lse_ref = oracle_sequence_fp8(inp, img, b, heads)
        o = got[b][:, heads]
        assert np.isfinite(o).all()
        assert np.abs(lse[b][:, heads] - lse_ref).max() <= LSE_MAX_ABS
        o_all.append(o), r_all.append(o_ref)
    o, r = np.concatenate(o_all), np.concatenate(r_all)
    assert np.abs(o - r).max() <= O_MAX_ABS and rel_l2(o, r) <= O_REL_L2, rel_l2(o, r)
