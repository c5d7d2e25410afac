"""A captured product of a matrix that is quantised again in place."""
import numpy as np
import pytest

import mx_util
from expert_util import device

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()


@pytest.mark.parametrize("own", [False, True])
def test_a_replayed_product_reads_the_scale_of_now(own):
    """Weights of which the library, or the caller, made the memory; the second ones are 64
    times as large, and so is the tensor scale that is found for them."""
    import torch

    import tma_pipelined_tensor_fp16_gb300 as tg
    rng = np.random.default_rng(3)
    w = device(rng.standard_normal((136, 256)).astype(np.float16))
    if own:
        W = tg.mx_quantize(w, "nvfp4")
    else:
        packed, scales, t, _ = mx_util.random_operand(rng, 136, 256, "nvfp4", False)
        W = tg.MXTensor.from_codes(device(packed), device(scales), 256, "nvfp4",
                                   torch.tensor([t], device="cuda"))
        tg.mx_quantize(w, "nvfp4", out=W)
    X = tg.mx_quantize(device(rng.standard_normal((40, 256)).astype(np.float16)), "nvfp4")
    plan = tg.MXPlan(40, 136, 256, format="nvfp4", out="f32")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        C = plan(X, W)
    for factor in (64.0, 1.0, 0.125):
        tg.mx_quantize(w * factor, "nvfp4", out=W)
        graph.replay()
        assert torch.equal(C, plan(X, W))
        assert torch.equal(C, plan(X, tg.mx_quantize(w * factor, "nvfp4")))
