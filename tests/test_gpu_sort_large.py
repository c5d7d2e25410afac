"""The sort of many slots over many experts: a cluster of more CTAs than the portable
eight, each with a full table of counts."""
import numpy as np
import pytest

from expert_util import device, sort_reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()


@pytest.mark.parametrize("tokens,topk,experts", [
    (9000, 1, 1024), (4100, 2, 1000), (25000, 4, 1024), (16385, 8, 513), (8193, 1, 600)])
def test_sort(tokens, topk, experts):
    import tma_pipelined_tensor_fp16_gb300 as tg
    rng = np.random.default_rng(tokens)
    ids = rng.integers(-3, experts + 3, (tokens, topk)).astype(np.int32)
    offsets, order, position = sort_reference(ids, experts)
    route = tg.ExpertRoute(tokens, topk, experts)
    for _ in range(2):
        route.sort(device(ids))
        assert (route.offsets.cpu().numpy() == offsets).all()
        assert (route.order.cpu().numpy() == order).all()
        assert (route.position.cpu().numpy() == position).all()


def test_first_sort_inside_a_capture():
    import torch

    import tma_pipelined_tensor_fp16_gb300 as tg
    rng = np.random.default_rng(7)
    ids = rng.integers(0, 900, (20000, 1)).astype(np.int32)
    dids = device(ids)
    route = tg.ExpertRoute(20000, 1, 900)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        route.sort(dids)
    graph.replay()
    torch.cuda.synchronize()
    assert (route.order.cpu().numpy() == sort_reference(ids, 900)[1]).all()
