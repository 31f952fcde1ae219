"""What the kernels of the 8-bit calls and of the write with the rotation promise in their
order of memory accesses, where no run can show it: a kernel started early sees its
predecessor's stores behind griddepcontrol.wait only."""
import re

import pytest

from test_q4_source import kernels


@pytest.mark.parametrize("source,count", [("rope_write.cu", 1), ("q8_cache.cu", 2),
                                          ("q8_decode.cu", 1), ("split.cuh", 1)])
def test_global_memory_is_read_behind_the_wait_only(source, count):
    found = kernels(source)
    assert len(found) == count
    for name, body in found.items():
        wait = re.search(r"griddepcontrol\.wait|PKV_DEPENDENT_PROLOGUE", body)
        assert wait, name
        before = body[:wait.start()]
        assert not re.search(r"__ldg|__ldcg|__ldcs|a\.\w+\s*\[|prefetch\.global", before), name
