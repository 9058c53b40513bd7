"""CPU checks of the binding itself: what it asks of torch, and what its typed
functions refuse."""
import ctypes
import os
import subprocess
import sys

import pytest

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


def test_paged_functions_take_their_own_structures_only():
    from flashattention_attention_b200 import fa
    d, pages, append, read, select = (fa.DecodeParams(), fa.KvPages(), fa.KvAppendRopeParams(), fa.KvReadParams(),
                                      fa.PageSelectParams())
    by = ctypes.byref
    for name, own, more in (("fa_attention_decode_paged", d, (None,)), ("fa_attention_decode_selected", d, (None, 1, None)),
                            ("fa_decode_pages_workspace_size", d, (0,)), ("fa_kv_append_rope_paged", append, (None,)),
                            ("fa_kv_read_paged", read, (None,)), ("fa_page_select", select, (None,))):
        fn = getattr(fa.lib, name)
        for bad in (by(fa.FwdParams()), by(pages), bytes(1000)):
            with pytest.raises(ctypes.ArgumentError):
                fn(bad, by(pages), *more)
        for bad in (by(own), bytes(1000)):
            with pytest.raises(ctypes.ArgumentError):
                fn(by(own), bad, *more)
        assert fn(None, None, *more) in (0, fa.FA_ERR_INVALID)  # the right types: the library's own checks answer
