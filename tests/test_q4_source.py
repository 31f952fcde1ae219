"""What the kernels on 4-bit pools promise in their order of memory accesses, where no
run can show it: a kernel started early sees its predecessor's stores behind
griddepcontrol.wait only."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(__file__), "..", "paged_kv_cache_70_gb300", "csrc")


def kernels(name):
    """{kernel: its body without comments} of a source file."""
    text = open(os.path.join(CSRC, name)).read()
    text = re.sub(r"//[^\n]*", "", text)
    out = {}
    for m in re.finditer(r"__global__ void[^;{]*?(\w+_kernel)\s*\([^{;]*\)\s*\{", text):
        depth, at = 1, m.end()
        while depth:
            depth += {"{": 1, "}": -1}.get(text[at], 0)
            at += 1
        out[m.group(1)] = text[m.end():at]
    return out


@pytest.mark.parametrize("source", ["q4_decode.cu", "q4_cache.cu", "compact.cu"])
def test_global_memory_is_read_behind_the_wait_only(source):
    found = kernels(source)
    assert found
    for name, body in found.items():
        wait = re.search(r"griddepcontrol\.wait|PKV_DEPENDENT_PROLOGUE", body)
        assert wait, name
        before = body[:wait.start()]
        assert not re.search(r"__ldg|__ldcg|__ldcs|a\.\w+\s*\[", before), name
