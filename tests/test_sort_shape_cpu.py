"""The launch of the expert sort, as the library computes it: every slot belongs to one
warp, in slot order, with 16 CTAs and with the 8 it falls back to, and the rows that
follow from the warps' counts are the stable sort's."""
import numpy as np
import pytest

from cpp_util import run_cpp
from expert_util import routing, sort_reference

SLOTS = [0, 1, 31, 128, 1023, 1024, 1025, 2049, 8192, 8193, 16384, 16385, 131072, 1 << 20, 1 << 30]


@pytest.fixture(scope="module")
def shapes(tmp_path_factory):
    """(slots, most CTAs) -> (CTAs, warps, run, bytes for 1024 experts)."""
    out = run_cpp(tmp_path_factory.mktemp("shape"), r"""
#include <cstdio>
#include <initializer_list>
#include "sort_shape.h"
int main()
{
    for (long long slots : {%s})
        for (int most : {8, 16}) {
            const tg::SortShape s = tg::sort_shape(slots, most);
            std::printf("%%lld %%d %%d %%d %%d %%u\n", slots, most, s.ctas, s.warps, s.run,
                        s.smem_bytes(1024));
        }
}
""" % ", ".join("%dLL" % s for s in SLOTS + [200, 1400, 12000]))
    rows = [tuple(map(int, line.split())) for line in out.splitlines()]
    return {r[:2]: r[2:] for r in rows}


def test_every_slot_has_a_warp(shapes):
    for (slots, most), (ctas, warps, run, smem) in shapes.items():
        assert 1 <= ctas <= most and ctas & (ctas - 1) == 0 and 8 <= warps <= 32
        assert run % 32 == 0 and ctas * warps * run >= slots
        assert smem <= 227 * 1024
        if slots > 1024 * most:
            assert ctas == most


@pytest.mark.parametrize("most", [8, 16])
@pytest.mark.parametrize("tokens,topk,experts", [(100, 2, 9), (700, 2, 9), (3000, 4, 33)])
def test_order_by_the_warps_counts(shapes, tokens, topk, experts, most):
    rng = np.random.default_rng(tokens)
    ids = routing(rng, tokens, topk, experts, 0.1)
    flat = ids.reshape(-1)
    ctas, warps, run, _ = shapes[flat.size, most]
    key = np.where((flat < 0) | (flat >= experts), experts, flat)
    counts = np.zeros((ctas * warps, experts + 1), dtype=int)
    for w in range(ctas * warps):
        np.add.at(counts[w], key[w * run:(w + 1) * run], 1)
    start = np.concatenate([[0], np.cumsum(counts.sum(0))[:-1]])
    at = start + np.cumsum(counts, 0) - counts
    position = np.empty(flat.size, dtype=int)
    for w in range(ctas * warps):
        for s in range(w * run, min((w + 1) * run, flat.size)):
            position[s] = at[w, key[s]]
            at[w, key[s]] += 1
    assert (position == sort_reference(ids, experts)[2].reshape(-1)).all()
