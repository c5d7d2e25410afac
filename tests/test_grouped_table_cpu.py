"""The grouped products' tile table for any offsets, as the kernel builds it: no more
tiles than the plan has counted on, no row in two of them, none outside the matrix."""
import re

import numpy as np
import pytest

from cpp_util import CSRC, run_cpp

HARNESS = r"""
#include <cstdint>
#include <cstdio>
#include <vector>
// One block of threads, run one after the other between its barriers: the functions of
// the kernel's table are compiled as they stand, with the warp's and the block's
// primitives over all threads at once.
struct GroupedParams { int rows, experts; const int* offsets; };
static const int GROUPED_THREADS = 192;
static int clamp_row(int r, int rows) { return r < 0 ? 0 : (r > rows ? rows : r); }
int main()
{
    int rows, experts, bm;
    while (std::scanf("%%d %%d %%d", &rows, &experts, &bm) == 3) {
        std::vector<int> offsets(experts + 1);
        for (int& o : offsets) if (std::scanf("%%d", &o) != 1) return 1;
        GroupedParams p = {rows, experts, offsets.data()};
        std::vector<int> row0(experts + 2), tile0(experts + 2);
        const int groups = p.experts + 1;
        const int share = (groups + GROUPED_THREADS - 1) / GROUPED_THREADS;
        auto start = [&](int g) { return %(start)s; };
        std::vector<int> sums(GROUPED_THREADS);
        int any = 0;
        for (int tid = 0; tid < GROUPED_THREADS; ++tid) {
            const int g0 = tid * share, BM = bm;
            (void)BM;
            %(first)s
            sums[tid] = sum;
            any |= descends;
        }
        int before = 0;
        for (int tid = 0; tid < GROUPED_THREADS; ++tid) {
            const int g0 = tid * share, BM = bm;
            const bool descends = any;
            (void)descends;
            int at = before;
            %(second)s
            before += sums[tid];
        }
        for (int g = 0; g < groups + 1; ++g) std::printf("%%d %%d ", row0[g], tile0[g]);
        std::printf("\n");
    }
}
"""


def _pieces():
    """The kernel's two loops and its reading of the offsets."""
    text = open(CSRC + "/kernel_grouped.cuh").read()
    body = text[text.index("void grouped_table("):]
    body = body[:body.index("\n}\n")]
    start = re.search(r"auto start = \[&\]\(int g\) \{ return (.*?); \};", body).group(1)
    first = body[body.index("int sum = 0;"):]
    first = first[:first.index("\n    }") + 6]
    second = body[body.index("for (int w = 0; w < warp"):]
    second = second[second.index("for (int i = 0;"):]
    second = second[:second.index("\n    }") + 6]
    if "descends" not in first:
        first += " const bool descends = false;"
    return dict(start=start, first=first, second=second)


def _tables(tmp_path):
    rng = np.random.default_rng(0)
    yield 4096, np.array([0, 4096] * 512 + [0])                     # up and down 1024 times
    yield 1 << 21, np.array([0, 1 << 21] * 512 + [0])
    yield 40, np.array([-5, 30, 10, 2 ** 31 - 1])
    for _ in range(40):
        experts = int(rng.integers(1, 1025))
        rows = int(rng.integers(1, 5000))
        table = rng.integers(-10, rows + 10, experts + 1)
        yield rows, table
        yield rows, np.sort(table)
        yield rows, np.concatenate([[0], np.sort(table)[1:]])


@pytest.mark.parametrize("bm", [128, 256])
def test_any_table(tmp_path, bm):
    cases = list(_tables(tmp_path))
    text = "".join("%d %d %d %s\n" % (rows, len(t) - 1, bm, " ".join(map(str, t.tolist())))
                   for rows, t in cases)
    (tmp_path / "in").write_text(text)
    source = HARNESS % _pieces()
    source = source.replace("int main()\n{", 'int main()\n{\n    if (!std::freopen("%s", "r", stdin)) '
                            "return 1;" % (tmp_path / "in"))
    lines = run_cpp(tmp_path, source).splitlines()
    assert len(lines) == len(cases)
    for (rows, table), line in zip(cases, lines):
        v = np.array(line.split(), dtype=np.int64).reshape(-1, 2)
        row0, tile0 = v[:, 0], v[:, 1]
        E = len(table) - 1
        assert 0 <= row0.min() and row0.max() <= rows and tile0[0] == 0
        counts = np.diff(tile0)
        assert (counts >= 0).all()
        assert tile0[-1] <= rows // bm + min(E + 1, rows)  # what the plan's limit allows for
        covered = np.diff(row0)
        assert (covered >= 0).all()  # so no row is in two groups
        assert (counts == -(-covered // bm)).all()
        inside = np.clip(table, 0, rows)
        if (np.diff(inside) >= 0).all():
            assert (row0[:E + 1] == inside).all()
