"""How the host reads a plan's device status record."""
from cpp_util import run_cpp


def test_reading_leaves_nothing_behind(tmp_path):
    """A CUDA graph repeats its run number with every replay, so a record that still
    names it as abandoned would make each later replay give up, silently."""
    out = run_cpp(tmp_path, r"""
#include <cstdio>
#include "gemm_common.h"
using namespace tg;
int main()
{
    DevStatus st = {};
    std::printf("%d\n", take_status(&st));
    st.code = DEV_TIMEOUT;
    st.where = WAIT_STALL;
    st.abort_epoch = 7;
    std::printf("%d\n", take_status(&st));
    std::printf("%d %d\n", st.code, st.abort_epoch);
    std::printf("%d\n", take_status(&st));
    st.abort_epoch = 9;  // a run that gave up without a code of its own
    std::printf("%d\n", take_status(&st));
    std::printf("%d\n", take_status(&st));
}
""")
    assert out.split("\n")[:-1] == ["0", "4", "0 0", "0", "4", "0"]
