"""The record of raised shared-memory limits: one per kernel and device."""
from cpp_util import run_cpp


def test_limits_belong_to_a_kernel_on_a_device(tmp_path):
    out = run_cpp(tmp_path, r"""
#include <cstdio>
#include "smem_limits.h"
int main()
{
    tg::SmemLimits limits;
    int a, b;  // two kernels
    limits.record(0, &a, 100000);
    std::printf("%d%d%d\n", limits.known(0, &a, 100000), limits.known(0, &a, 100001),
                limits.known(0, &b, 1));
    std::printf("%d\n", limits.known(1, &a, 1));
    limits.record(1, &a, 50000);
    limits.record(0, &a, 60000);  // never lowered
    std::printf("%d%d%d\n", limits.known(0, &a, 100000), limits.known(1, &a, 50000),
                limits.known(1, &a, 50001));
}
""")
    assert out.split("\n")[:-1] == ["100", "0", "110"]


def test_the_current_device_is_part_of_the_key():
    import os

    from cpp_util import CSRC
    text = open(os.path.join(CSRC, "launch.h")).read()
    body = text[text.index("cudaError_t ensure_smem_limit"):]
    body = body[:body.index("\n}")]
    assert "cudaGetDevice" in body
    assert body.count("(device, key, bytes)") == 2
