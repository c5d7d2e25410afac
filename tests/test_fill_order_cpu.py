"""Memory that a plan's creator fills is filled when it returns: the first run may come at once
on a stream that waits for nothing else.  A copy that has not landed goes wrong only when the
two meet, and then through addresses that are not there yet, so the sources are read as text."""
import os
import re

import pytest

from cpp_util import CSRC


def _source(name):
    return re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())


def test_a_fill_is_waited_for():
    """On a stream that waits for no other one, on which nothing else runs."""
    body = _source("runtime.cu")
    body = body[body.index("cudaError_t fill_memory("):]
    body = body[:body.index("\n}")]
    order = [body.index(s) for s in ("cudaStreamNonBlocking", "cudaMemcpyAsync(", "cudaMemsetAsync(",
                                     "cudaStreamSynchronize(stream)", "return e != cudaSuccess")]
    assert order == sorted(order)
    assert len(re.findall(r"\breturn\b", body[order[1]:order[3]])) == 0


@pytest.mark.parametrize("file", ["api.cu", "clip.cu", "grouped.cu", "mx_plan.cu", "w4.cu"])
def test_creators_fill_through_it(file):
    text = _source(file)
    plain = re.findall(r"\bcudaMem(?:cpy|set)\([^;]*;", text)
    assert all("cudaMemcpyDeviceToHost" in call for call in plain)
    assert "fill_memory(" in text


def test_a_records_clearing_is_waited_for():
    """The next run may have ended with a status of its own before a late clearing."""
    body = _source("runtime.cu")
    body = body[body.index("int read_device_status("):]
    assert "cudaMemcpyHostToDevice" not in body and "fill_memory(record" in body
