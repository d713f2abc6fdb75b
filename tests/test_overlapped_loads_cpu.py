"""Kernels that are launched early may be resident while kernels two or three
places ahead of them in the stream still write: what those write is read by
coherent loads.  The non-coherent ones (ld.global.nc, __ldg, ldg16) are for what
no such kernel writes."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "long_context_emitting_b200", "csrc")

# file, the overlapped kernels' part of it, what may be read without coherence there
PARTS = [
    ("cache_q4.cu", "", ()),
    ("decode_q4.cu", "", ()),
    ("norm_rope.cu", "", ("ldg16(a.w[part]",)),                  # norm weights
    # the 16-bit gather kernel: selected indices, which Top-k writes, a kernel that is waited for in full
    ("decode.cu", "decode_gather_kernel(const SplitArgs", ("__ldg(rows",)),
]


@pytest.mark.parametrize("name,start,allowed", PARTS, ids=[p[0] for p in PARTS])
def test_no_read_only_loads_of_what_kernels_write(name, start, allowed):
    text = open(os.path.join(CSRC, name)).read()
    text = re.sub(r"//[^\n]*", "", text[text.index(start):])
    assert "overlap_launches()" in text or "grid_dependency_wait()" in text
    for a in allowed:
        text = text.replace(a, "")
    found = re.findall(r"(?:__ldg|ldg16|ldg_stream16)\([^;]*;|[^;]*\.nc[.\w]*[^;]*;", text)
    assert not found, found
