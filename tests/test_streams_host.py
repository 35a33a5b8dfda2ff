"""What a call allocates or fills itself belongs to the stream it launches on: checked without a GPU, with the
library, the streams and the address checks replaced by recorders and every torch operation logged with the
stream it would have been issued on."""

import contextlib

import pytest
import torch
from torch.utils._python_dispatch import TorchDispatchMode

CURRENT, SIDE = 11, 22  # stream handles


class Recorder(TorchDispatchMode):
    """Logs ("torch", operation, stream), ("launch", function, stream) and waits in the order they happen."""

    def __init__(self):
        super().__init__()
        self.stack, self.log = [CURRENT], []

    def __torch_dispatch__(self, func, types, args=(), kwargs=None):
        self.log.append(("torch", func.overloadpacket.__name__, self.stack[-1]))
        return func(*args, **(kwargs or {}))

    def streams_of(self, *names):
        return {s for kind, name, s in self.log if kind == "torch" and name in names}


class Stream:
    """A torch stream, as far as the package uses one."""

    rec = None

    def __init__(self, handle, device=None):
        assert handle not in (0, 1)  # no handle of a stream that ExternalStream can wrap
        self.handle = self.cuda_stream = handle

    def wait_stream(self, other):
        self.rec.log.append(("wait", other.handle, self.handle))

    def synchronize(self):
        self.rec.log.append(("synchronize", "", self.handle))


class Lib:
    """The library: a launch is logged with its last argument, a size query goes to the real one."""

    def __init__(self, rec, real):
        self.rec, self.real = rec, real

    def __getattr__(self, name):
        if name.endswith("_size") or name.endswith("_path") or name.endswith("_splits"):
            return getattr(self.real, name)

        def launch(*args):
            self.rec.log.append(("launch", name, args[-1]))
            return 0
        return launch


@pytest.fixture
def rec(monkeypatch):
    from mla_absorbed_decode_absorb_gb300 import ops
    rec = Recorder()

    @contextlib.contextmanager
    def stream(s):
        rec.stack.append(s.handle)
        try:
            yield
        finally:
            rec.stack.pop()

    fake = type("FakeStream", (Stream,), {"rec": rec})
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", fake)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: fake(rec.stack[-1]))
    monkeypatch.setattr(ops, "lib", Lib(rec, ops.lib))
    monkeypatch.setattr(ops, "mla_linear_strided", lambda *a, stream=None: rec.log.append(  # asks its y for a CUDA tensor
        ("launch", "mla_linear_strided", rec.stack[-1] if len(a) < 8 or a[7] is None else int(a[7]))))
    monkeypatch.setattr(ops, "_device", lambda: -1)
    monkeypatch.setattr(ops, "_dev", lambda t, *a, **k: t.data_ptr())
    monkeypatch.setattr(ops, "_dev_or_pinned", lambda t, *a, **k: t.data_ptr())
    monkeypatch.setattr(ops, "_stream", lambda s, device=None: rec.stack[-1] if s is None else int(s))
    return rec


def fp8_cache(pages):
    return (torch.zeros(pages, 64, 512, dtype=torch.uint8), torch.zeros(pages, 64),
            torch.zeros(pages, 64, 64, dtype=torch.float16))


@pytest.mark.parametrize("stream,where", [(None, CURRENT), (SIDE, SIDE)])
def test_read_back_fills_its_rows_on_the_stream_it_reads_on(rec, stream, where):
    """Filled on the current stream while the read runs on another, the sentinel could land over the rows read back."""
    from mla_absorbed_decode_absorb_gb300 import ops
    cache, table = fp8_cache(3), torch.zeros(2, 2, dtype=torch.int32)
    lens = torch.tensor([70, 100], dtype=torch.int32)
    with rec:
        rows = ops.mla_read_kv_fp8(cache, table, lens, 100, stream=stream)
    assert rows.shape == (4, 64, 576) and torch.isnan(rows.float()).all()
    assert ("launch", "mla_read_kv_fp8", where) in rec.log
    assert rec.streams_of("full", "fill_", "empty") == {where}


def one_stream(rec, where):
    """Everything in the log ran on ``where``, behind what the current stream held, and was waited for at the end."""
    kinds = [k for k, _, _ in rec.log]
    assert {s for k, _, s in rec.log if k in ("torch", "launch")} == {where}
    if where != CURRENT:
        assert rec.log[0] == ("wait", CURRENT, where)
    assert rec.log[-1] == ("synchronize", "", where)
    assert "launch" in kinds


@pytest.mark.parametrize("stream,where", [(None, CURRENT), (SIDE, SIDE)])
@pytest.mark.parametrize("n_q,cache_format", [(70, "fp8"), (70, "bf16"), (2, "bf16"), (2, "fp8")])
def test_a_decode_session_is_laid_out_on_one_stream(rec, stream, where, n_q, cache_format):
    """The pools' fills, the history's copies, the appends and the page table of the rows read back: on two streams the
    appends would not wait for the fills, a step could read a table that is not written yet, and the memory of one
    sequence's history could be taken for the next one's while the append still reads it."""
    from mla_absorbed_decode_absorb_gb300 import workloads as W
    from mla_absorbed_decode_absorb_gb300.runtime import DecodeSession
    inp = W.generate(W.custom("streams", [0, 63, 130], n_q=n_q, cache_format=cache_format), seed=3)
    with rec:
        s = DecodeSession(inp, device="cpu", stream=stream)
    assert s.path == ("non_absorbed" if n_q == 70 else "absorbed")
    one_stream(rec, where)


@pytest.mark.parametrize("stream,where", [(None, CURRENT), (SIDE, SIDE)])
@pytest.mark.parametrize("kind", ["plain", "fold", "few_bits"])
def test_a_layer_session_is_laid_out_on_one_stream(rec, stream, where, kind):
    """... and its weights: quantised or folded from tensors that are given back while the launches still read them."""
    from mla_absorbed_decode_absorb_gb300 import workloads as W
    from mla_absorbed_decode_absorb_gb300.runtime import LayerNorms, LayerSession
    li = W.generate_layer(W.Workload("streams", batch=2, n_q=2, lengths=(0, 70), d_model=256), seed=3)
    kw = {"plain": {}, "fold": dict(fold=True)}.get(kind)
    if kw is None:
        ones = [torch.ones(n, dtype=torch.bfloat16) for n in (256, W.D_Q_LATENT, W.D_LATENT)]
        kw = dict(weights="w4", activations="fp8", norms=LayerNorms(*ones), residual=li.x.clone())
    with rec:
        LayerSession(li, device="cpu", stream=stream, **kw)
    one_stream(rec, where)


def test_raw_handles_of_streams(monkeypatch):
    """A handle is an external stream; 0 and 1 (the legacy default stream), which torch does not take for one, are its
    default stream."""
    from mla_absorbed_decode_absorb_gb300 import ops
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: ("external", handle))
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: "default")
    assert ops._torch_stream(SIDE) == ("external", SIDE)
    assert ops._torch_stream(0) == ops._torch_stream(1) == "default"


def calls():
    """Every call that makes an output or a workspace when it is given none: (name, arguments)."""
    bf, i32 = torch.bfloat16, torch.int32

    def z(*shape, dtype=bf):
        return torch.zeros(*shape, dtype=dtype)
    T, K, N = 3, 4096, 64  # K split: the bf16 projections take a workspace
    w4 = (z(N, K // 2, dtype=torch.uint8), z(N, K // 128))
    lens, table, cache = z(1, dtype=i32), z(1, 2, dtype=i32), z(2, 64, 576)
    heads, rope = z(128, 128, 512), z(8, 64, dtype=torch.float32)
    q, qr, prior = z(1, 1, 128, 128), z(1, 1, 128, 64), z(1, dtype=i32)
    q_abs, o = z(1, 1, 128, 576), z(1, 1, 128, 512, dtype=torch.float32)
    kv = z(1, 128, 100, 128)
    x8, sx = z(T, K, dtype=torch.uint8), z(T, K // 128, dtype=torch.float32)
    return [
        ("mla_rms_norm", (z(T, K), z(K))), ("mla_rms_norm_fp8", (z(T, K), z(K))),
        ("mla_quantize_w4", (z(N, K),)), ("mla_dequantize_w4", w4),
        ("mla_linear_w4", (z(T, K), *w4)), ("mla_linear_w4_fp8", (x8, sx, *w4)),
        ("mla_linear_w4_pair", (z(T, K), w4, w4)), ("mla_linear_w4_fp8_pair", (x8, sx, w4, w4)),
        ("mla_read_kv_fp8", (fp8_cache(2), table, lens, 100)),
        ("rope_table", (8, "cpu")), ("mla_linear", (z(T, K), z(N, K))),
        ("mla_linear_pair", (z(T, K), z(N, K), z(N, K))),
        ("mla_absorb_q", (q, qr, prior, heads, rope)),
        ("mla_decode_attn", (q_abs, cache, table, lens, 1, 100)),
        ("mla_out_absorb", (o, heads)),
        ("mla_combine_out_absorb", (1, 1, 100, 0, z(16, dtype=torch.uint8), None, heads)),
        ("mla_decompress_kv", (cache, table, lens, 100, heads, heads)),
        ("mla_prefill_attn", (q, qr, prior, rope, kv, kv, cache, table, lens)),
    ]


@pytest.mark.parametrize("stream,where", [(None, CURRENT), (SIDE, SIDE)])
@pytest.mark.parametrize("name,args", [pytest.param(*c, id=c[0]) for c in calls()])
def test_what_a_call_makes_belongs_to_its_stream(rec, monkeypatch, stream, where, name, args):
    """Memory taken on the current stream may have been given back there by work that is still running, and its next
    user there does not wait for the launch.  What the caller gets is held for the current stream too."""
    from mla_absorbed_decode_absorb_gb300 import ops
    held = []
    monkeypatch.setattr(torch.Tensor, "is_cuda", True)
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: held.append((t.data_ptr(), s.handle)))
    with rec:
        out = getattr(ops, name)(*args, stream=stream)
    assert rec.log[-1][::2] == ("launch", where)
    assert rec.streams_of("empty", "empty_strided", "empty_like", "full") == {where}
    made = [t for t in (out if isinstance(out, tuple) else (out,)) if t is not None]
    assert sorted(held) == ([] if stream is None else sorted((t.data_ptr(), CURRENT) for t in made))
