"""Which tile counter a grouped product's run uses: never one that another run on the
GPU may be using."""
from cpp_util import run_cpp


def test_runs_that_may_overlap_have_counters_of_their_own(tmp_path):
    out = run_cpp(tmp_path, r"""
#include <cstdio>
#include <set>
#include "counter_slots.h"
using tg::CounterSlots;
int main()
{
    CounterSlots s;
    bool over = false, any = false;
    std::set<int> used;
    for (int id = 1; id <= CounterSlots::STREAMS; ++id) {
        const int slot = s.of_stream(1000 + id, &over);
        used.insert(slot);
        any |= over || slot < 0 || slot >= CounterSlots::STREAMS;
    }
    std::printf("%d %d\n", static_cast<int>(used.size()), any);
    // a stream keeps its own
    const int a = s.of_stream(1001, &over), b = s.of_stream(1001, &over);
    std::printf("%d %d\n", a == b, over);
    // one stream more takes over the one unused for longest, 1002, and says so
    const int c = s.of_stream(9999, &over);
    std::printf("%d %d\n", c == 1, over);
    s.of_stream(9999, &over);
    std::printf("%d\n", over);
    s.give_up(7);  // then it is the next to be taken over
    const int d = s.of_stream(10000, &over);
    std::printf("%d %d\n", d, over);
    // captured launches: each its own, none of a stream's, until all are held
    used.clear();
    for (int i = 0; i < CounterSlots::CAPTURES; ++i) used.insert(s.of_capture());
    std::printf("%d %d\n", static_cast<int>(used.size()), *used.begin());
    std::printf("%d\n", s.of_capture());
    s.release(300);  // a graph is gone
    const int again = s.of_capture(), none = s.of_capture();
    std::printf("%d %d\n", again, none);
    std::printf("%d\n", *used.rbegin() < CounterSlots::COUNT);
}
""")
    assert out.split("\n")[:-1] == ["256 0", "1 0", "1 1", "0", "7 1", "65280 256", "-1",
                                    "300 -1", "1"]


def test_the_plan_asks_for_its_run_s_counter():
    """No run takes a counter without asking whose it is."""
    import os

    from cpp_util import CSRC
    text = open(os.path.join(CSRC, "grouped.cu")).read()
    run = text[text.index("int gemm_grouped_run("):text.index("int gemm_grouped_get_device_status")]
    assert "counter_of(pool.slots, stream, &slot)" in run and "+ slot;" in run
