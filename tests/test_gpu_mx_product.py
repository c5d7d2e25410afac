"""Block-scaled products: sums that fp32 holds bit for bit, random ones within the
tolerance of expert_util (the products themselves are exact)."""
import numpy as np
import pytest

import mx_util
from expert_util import assert_same, assert_within, device, tolerance

pytestmark = pytest.mark.gpu

FORMATS = ["mxfp8", "mxfp4", "nvfp4"]


@pytest.fixture(scope="module", autouse=True)
def _built():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()


def _operand(rng, rows, K, format, exact):
    import torch

    import tma_pipelined_tensor_fp16_gb300 as tg
    packed, scales, t, v = mx_util.random_operand(rng, rows, K, format, exact)
    scale = torch.tensor([t], device="cuda") if format == "nvfp4" and t != 1.0 else None
    return tg.MXTensor.from_codes(device(packed), device(scales), K, format, scale), v


def _run(M, N, K, format, out, exact, seed=0, **options):
    import torch

    import tma_pipelined_tensor_fp16_gb300 as tg
    rng = np.random.default_rng(M * 31 + N * 7 + K + seed)
    A, a = _operand(rng, M, K, format, exact)
    B, b = _operand(rng, N, K, format, exact)
    plan = tg.MXPlan(M, N, K, format=format, out=out, **options)
    C = torch.full((M + 1, N), float("nan"), dtype=plan.dtype, device="cuda")
    plan(A, B, C[:-1])
    torch.cuda.synchronize()
    assert plan.device_status() == 0, tg.gemm_last_error() + "; " + plan.describe()
    assert torch.isnan(C[-1]).all(), "wrote past the end"
    return C[:-1].cpu().numpy(), a @ b.T, np.abs(a) @ np.abs(b).T, plan.describe()


SINGLE = [  # M, N, K, split
    (1, 8, 8, 1), (1, 16, 64, 1), (1, 128, 128, 0), (3, 136, 256, 1), (16, 256, 512, 2),
    (17, 72, 1000, 1), (32, 264, 2048, 4), (33, 520, 1032, 2), (64, 128, 4096, 8),
    (65, 128, 256, 1), (100, 200, 520, 2), (128, 128, 1024, 1), (129, 136, 264, 1),
    (300, 392, 2056, 4), (1, 1000, 8192, 0), (5, 2048, 96, 0), (200, 64, 32, 0),
]


@pytest.mark.parametrize("format", FORMATS)
@pytest.mark.parametrize("M,N,K,split", SINGLE)
def test_single_exact(M, N, K, split, format):
    for out in ("f32", "f16"):
        got, ref, _, what = _run(M, N, K, format, out, True, kernel="single", split=split)
        assert_same(got, ref, out, what)


PAIR = [(1, 8, 8), (128, 128, 64), (256, 256, 256), (257, 264, 520), (100, 1000, 136),
        (1000, 520, 2056), (512, 4096, 1024), (130, 300 // 4 * 4 + 4, 4096)]


@pytest.mark.parametrize("format", FORMATS)
@pytest.mark.parametrize("M,N,K", PAIR + [(600, 1100, 4096), (2000, 2048, 520)])
def test_pair_exact(M, N, K, format):
    for out in ("f32", "f16"):
        if N % 8 and out == "f16":
            continue
        got, ref, _, what = _run(M, N, K, format, out, True, kernel="pair")
        assert_same(got, ref, out, what)


@pytest.mark.parametrize("format", FORMATS)
@pytest.mark.parametrize("M,N,K", [(4900, 2568, 264), (5004, 2312, 1536), (4640, 2824, 1544)])
def test_pair_many_tiles(M, N, K, format):
    """Several tiles a cluster, some of whose warps have no rows to store, between full ones."""
    for out in ("f32", "f16"):
        got, ref, _, what = _run(M, N, K, format, out, True, kernel="pair")
        assert_same(got, ref, out, what)


@pytest.mark.parametrize("format", FORMATS)
@pytest.mark.parametrize("M,N,K,options", [
    (7, 264, 4096, {}), (64, 512, 2048, {}), (300, 520, 1000, {}),
    (600, 776, 1500 // 4 * 4, {"kernel": "pair"}), (1, 1024, 16384, {})])
def test_random_values(M, N, K, options, format):
    for out in ("f32", "f16"):
        got, ref, size, what = _run(M, N, K, format, out, False, **options)
        if out == "f16":
            fits = np.abs(ref) < 60000
            assert fits.mean() > 0.5
            got, ref, size = got[fits], ref[fits], size[fits]
        assert_within(got, ref, tolerance(ref, size, K, out), what)
