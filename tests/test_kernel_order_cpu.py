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


def _orders(ops):
    """The orders in which one thread's operations may take effect: program order for
    operations on one address and across a fence, any order otherwise."""
    for p in itertools.permutations(range(len(ops))):
        place = {i: k for k, i in enumerate(p)}
        if all(place[i] < place[j] for i in range(len(ops)) for j in range(i + 1, len(ops))
               if ops[i][1] == ops[j][1] or "fence" in (ops[i][0], ops[j][0])):
            yield [ops[i] for i in p]


def _merges(a, b):
    if not a or not b:
        yield list(a) + list(b)
        return
    for rest in _merges(a[1:], b):
        yield [a[0]] + rest
    for rest in _merges(a, b[1:]):
        yield [b[0]] + rest


def _left_over(take, done, fence):
    """Whether some order leaves tiles counted as taken after two CTAs have each taken
    two tiles and arrived, the last one setting the counters back."""
    cta = [("take", take), ("take", take)] + ([("fence", None)] if fence else []) + \
        [("done", done)]
    for x, y in itertools.product(list(_orders(cta)), repeat=2):
        for order in _merges([(0,) + o for o in x], [(1,) + o for o in y]):
            taken = arrived = 0
            for _, op, _addr in order:
                if op == "take":
                    taken += 1
                elif op == "done":
                    arrived += 1
                    if arrived == 2:
                        taken = 0
            if taken:
                return True
    return False


@pytest.mark.parametrize("file", ["kernel_grouped.cuh", "kernel_grouped_pair.cuh"])
def test_tile_counter_starts_every_run_at_zero(file):
    """Tiles are handed out from a counter that the last CTA to finish sets back.  A
    tile taken must not be counted after that."""
    text = _source(file)
    if "grouped_take(p.counter)" in text:  # through the functions of kernel_grouped.cuh
        assert len(re.findall(r"grouped_(?:take|finish)\(p\.counter", text)) == 2
        text = _source("kernel_grouped.cuh")
    calls = re.findall(r"atomicAdd\(\s*([^,]+?)\s*,", text)
    assert len(calls) == 2, calls
    take, done = calls
    at = text.index("atomicAdd(" + take)
    fence = "__threadfence" in text[at:text.index("atomicAdd(" + done, at + 1)]
    assert not _left_over(take, done, fence)


def test_the_model_finds_a_late_count():
    assert _left_over("a", "b", False)
    assert not _left_over("a", "b", True)
    assert not _left_over("a", "a", False)


@pytest.mark.parametrize("file", ["kernel_ws.cu", "kernel_ws2.cuh", "kernel_grouped.cuh",
                                  "kernel_grouped_pair.cuh", "w4.cu"])
def test_copies_in_flight_are_waited_for_whoever_gave_up(file):
    """A producer that issued all its copies may end before any wait of its own fails,
    while the role that reads them has given up: its drain must not depend on its own
    state."""
    for _, name, body in _kernels():
        if _ != file:
            continue
        for m in re.finditer(r"wd\.drain\(bar(?:_addr)?\([^;]*?(?:FULL|TAIL)", body):
            depth, conditions = 0, []
            for line in reversed(body[:m.start()].split("\n")):
                depth += line.count("{") - line.count("}")
                if depth > len(conditions):
                    conditions.append(line.strip())
                if "warp == 0" in line or "warp < 10" in line:
                    break
            assert not any("aborted" in c for c in conditions), (name, conditions)


def test_a_relaxed_arrival_follows_the_use_of_what_was_read():
    """A reader gives a tile's slot back with a relaxed arrival, which orders nothing by
    itself: the value must have been used before (the instruction that uses it waits for
    the load, and instructions issue in order), and no other lane may still be reading."""
    text = _source("kernel_grouped_pair.cuh")
    body = text[text.index("int pair_read("):]
    body = body[:body.index("\n}\n")]
    load, use, arrive = (body.index(s) for s in ("ld_shared_int(", "__shfl_sync(",
                                                 "mbar_arrive_cluster_relaxed("))
    assert load < use < arrive
    assert "lane == 0" in body[:load].split(";")[-1]  # the others take it from lane 0
