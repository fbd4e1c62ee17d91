"""Kernels launched with programmatic serialization are on the GPU while the kernel before them still writes.  A load
through the read-only path (__ldg, ld.global.nc) asks that its data stay unchanged for as long as the reading kernel
lives, so such kernels take it only for weights, which no kernel of the library writes; queries, caches, scales,
scores and thresholds go through ordinary loads after the dependency wait."""
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "long_context_decoding_saga_b200", "csrc")

# file: what its read-only loads may be of (the weights of the norms and of the QKV projection)
WEIGHTS = {"saga_cache.cu": ("wp + c * 8",), "saga_kernels.cu": ("wrow + k0",), "saga_tree.cu": ()}


@pytest.mark.parametrize("name", sorted(WEIGHTS))
def test_only_weights_are_read_through_the_read_only_path(name):
    src = open(os.path.join(CSRC, name)).read()
    assert "pdl_wait();" in src
    code = re.sub(r"//[^\n]*", "", src)
    assert "ld.global.nc" not in code and "__restrict__" not in code
    loads = re.findall(r"__ldg\(([^;]*);", code)
    assert all(any(w in x for w in WEIGHTS[name]) for x in loads), loads
