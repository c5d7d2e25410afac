"""Sizes whose tile coordinates would pass 2^31 are refused before anything is
allocated: the kernels add up to a tile's width to a coordinate in 32 bits."""
import pytest

EDGE = (1 << 31) - 65536  # the largest size that is taken, where nothing else limits it


@pytest.fixture(scope="module")
def b():
    from tma_pipelined_tensor_fp16_gb300 import binding, build
    build.build()
    return binding


def _grouped(b, rows, N, K, experts=1, op=0):
    assert not b.lib().gemm_grouped_create_plan(rows, N, K, experts, op, 1)
    return b.gemm_last_status()


def _w4(b, M, N, K, experts=0):
    assert not b.lib().gemm_w4_create_plan(M, N, K, 32, experts, 1, 1)
    return b.gemm_last_status()


@pytest.mark.parametrize("op", [0, 1, 2])
def test_grouped(b, op):
    import torch
    over = (1 << 31) - 8
    for shape in ((over, 8, 8), (8, over, 8), (8, 8, over)):
        assert _grouped(b, *shape, op=op) == b.GEMM_ERR_INVALID_ARG
    assert _grouped(b, 8, over // 16 * 8, 8, experts=2, op=op) == b.GEMM_ERR_UNSUPPORTED
    if not torch.cuda.is_available():  # taken, up to the device check
        assert _grouped(b, EDGE, 8, 8, op=op) == b.GEMM_ERR_NO_DEVICE
        assert _grouped(b, 8, EDGE, 8, op=op) == b.GEMM_ERR_NO_DEVICE


def test_w4(b):
    import torch
    over = (1 << 31) - 8
    assert _w4(b, 1, over, 32) == b.GEMM_ERR_INVALID_ARG
    assert _w4(b, over, 8, 32) == b.GEMM_ERR_INVALID_ARG
    assert _w4(b, 1, 8, (1 << 31) - 32) == b.GEMM_ERR_INVALID_ARG
    assert _w4(b, 1, over // 16 * 8, 32, experts=2) == b.GEMM_ERR_UNSUPPORTED
    if not torch.cuda.is_available():
        assert _w4(b, 1, EDGE, 32) == b.GEMM_ERR_NO_DEVICE
