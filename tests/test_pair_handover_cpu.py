"""The block-scaled pair kernel gives an accumulator back with a relaxed arrival, which orders
nothing by itself: one lane arrives for a warp whose reads have completed in every lane, and the
next MMAs come behind a wait and a fence.  Read as text: nothing here runs on a device."""
import os
import re

from cpp_util import CSRC


def test_reads_are_complete_before_the_arrival():
    text = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, "mx_pair.cu")).read())
    load = text[text.index("void tmem_load_64cols("):]
    load = load[:load.index("\n}\n")]
    assert load.index("tcgen05.ld.sync.aligned") < load.index("tcgen05.wait::ld.sync.aligned")
    assert '"+r"(r[i])::"memory"' in load[load.index("wait::ld"):]  # nothing is read before it
    body = text[text.index("k_mx_pair("):]
    read = body.index("tmem_load_64cols(taddr + col, v)")
    order = [body.index(s, read) for s in ("tc_fence_before_sync()", "__syncwarp()",
                                           "if (lane == 0) mbar_arrive_cluster_relaxed(to_leader)")]
    assert read < order[0] and order == sorted(order)
    issue = body[body.index("WAIT_TMEM_EMPTY"):]
    assert issue.index("tc_fence_after_sync()") < issue.index("copy_scales<true>(") \
        < issue.index("mx_mma_k96_pair(")
