"""A plan beside none is refused."""
import pytest


@pytest.fixture(scope="module")
def b():
    from tma_pipelined_tensor_fp16_gb300 import binding, build
    build.build()
    return binding


def test_no_plan(b):
    assert not b.lib().gemm_mx_create_plan_beside(None, 8, 8, 64, 1, 0, 0)
    assert b.gemm_last_status() == b.GEMM_ERR_INVALID_ARG
