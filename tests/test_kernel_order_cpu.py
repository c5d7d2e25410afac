"""The order of a few operations in the kernels' sources that no run on a GPU
shows reliably, because a wrong order goes wrong only when two memory operations
or two kernels happen to meet.  Read as text: nothing here runs on a device."""
import glob
import itertools
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "tma_pipelined_tensor_fp16_gb300", "csrc")


def _source(name):
    text = open(os.path.join(CSRC, name)).read()
    return re.sub(r"//[^\n]*", "", text)


def _kernels():
    """(file, kernel, body) of every __global__ function."""
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu*"))):
        text = _source(os.path.basename(path))
        for part in re.split(r"(?=__global__)", text)[1:]:
            name = re.search(r"\b(k_\w+)\s*\(", part).group(1)
            yield os.path.basename(path), name, part[part.index("{"):]


def test_tensor_memory_is_allocated_before_dependents_start():
    """A dependent kernel that starts on the same SM may take the rest of tensor memory
    and wait for this kernel to end; an allocation after that would wait for ever."""
    seen = 0
    for file, name, body in _kernels():
        alloc = [m.start() for m in re.finditer(r"\btmem_alloc(_pair)?\(", body)]
        trigger = [m.start() for m in re.finditer(r"\bgriddep_launch_dependents\(", body)]
        if alloc and trigger:
            seen += 1
            assert max(alloc) < min(trigger), "%s: %s triggers before it allocates" % (file, name)
    assert seen >= 4
