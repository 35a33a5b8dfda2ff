"""The Python bindings without a GPU."""

import os
import subprocess
import sys

CODE = """
import torch
for name in ("_cuda_getDevice", "_cuda_getCurrentRawStream"):
    if hasattr(torch._C, name):
        delattr(torch._C, name)
from mla_absorbed_decode_absorb_gb300 import ops
torch.cuda.init = lambda: None
torch.cuda.current_device = lambda: 3
torch.cuda.current_stream = lambda device=None: type("S", (), {"cuda_stream": 100 + device})()
assert ops._device() == 3 and ops._stream(None) == 103 and ops._stream(None, 5) == 105
print("imported")
"""


def test_bindings_import_without_torch_internals():
    """The quick ways to the current device and stream are taken where torch has them; without them (a torch built
    without CUDA) the package is imported all the same and asks the public functions."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", CODE], cwd=root, capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and "imported" in r.stdout, r.stderr[-2000:]
