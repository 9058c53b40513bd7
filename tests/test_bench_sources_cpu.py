"""CPU check that the bench keys a kernel's committed DRAM traffic by every file
that holds its device code."""
import os
import re

import bench

CSRC = os.path.join(os.path.dirname(os.path.abspath(bench.__file__)), "flashattention_attention_b200", "csrc")


def _device_headers(name, seen):
    """The .cuh files that csrc/<name> includes, directly or through another file of csrc."""
    with open(os.path.join(CSRC, name)) as f:
        for inc in re.findall(r'#include "([^"]+)"', f.read()):
            if os.path.exists(os.path.join(CSRC, inc)) and inc not in seen:
                seen.add(inc)
                _device_headers(inc, seen)
    return {s for s in seen if s.endswith(".cuh")}


def test_traffic_is_keyed_by_every_device_header():
    for kernel, files in bench.KERNEL_SOURCES.items():
        want = _device_headers(files[0], set())
        assert want <= set(files), (kernel, want - set(files))
