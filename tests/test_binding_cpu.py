"""CPU checks of the binding itself: what it asks of torch, and what its typed
functions refuse."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_import_needs_no_private_names_of_torch():
    """A torch built without CUDA has no accessors of the device and the stream: the module imports, and its host
    functions work."""
    code = ("import torch\n"
            "for name in ('_cuda_getDevice', '_cuda_getCurrentRawStream'):\n"
            "    if hasattr(torch._C, name): delattr(torch._C, name)\n"
            "from flashattention_attention_b200 import fa\n"
            "print(tuple(fa.rope_table(3, 16).shape))\n")
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "(3, 16)", r.stderr[-2000:]
