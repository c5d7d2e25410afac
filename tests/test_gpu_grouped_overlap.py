"""Runs of one grouped plan that overlap on the GPU: on two streams, and a graph's
replays beside eager calls.  Whole numbers, bit for bit."""
import numpy as np
import pytest

from expert_util import device, integers, offsets_of

pytestmark = pytest.mark.gpu

ROWS, N, K, EXPERTS = 900, 1032, 200, 5


@pytest.fixture(scope="module", autouse=True)
def _built():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()


def _inputs(rng):
    counts = rng.multinomial(ROWS, np.ones(EXPERTS) / EXPERTS)
    offsets = offsets_of(counts)
    A, B = integers(rng, (ROWS, K)), integers(rng, (EXPERTS, N, K))
    want = np.concatenate([A[offsets[e]:offsets[e + 1]].astype(np.float64) @
                           B[e].astype(np.float64).T for e in range(EXPERTS)])
    return device(A), device(B), device(offsets), device(want.astype(np.float16))


@pytest.mark.parametrize("tile", ["128x128", "128x256", "256x256"])
def test_two_streams(tile):
    import torch

    import tma_pipelined_tensor_fp16_gb300 as tg
    rng = np.random.default_rng(4)
    plan = tg.GroupedPlan(ROWS, N, K, EXPERTS, tile=tile)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    inputs = [_inputs(rng), _inputs(rng)]
    outs = [[torch.full((ROWS, N), float("nan"), dtype=torch.float16, device="cuda")
             for _ in range(40)] for _ in streams]
    torch.cuda.synchronize()
    for i in range(40):
        for s, (A, B, offsets, _), out in zip(streams, inputs, outs):
            plan(A, B, offsets, out[i], stream=s)
    torch.cuda.synchronize()
    assert plan.device_status() == 0
    for (_, _, _, want), out in zip(inputs, outs):
        for C in out:
            assert torch.equal(C, want)


def test_replay_beside_eager_calls():
    import torch

    import tma_pipelined_tensor_fp16_gb300 as tg
    rng = np.random.default_rng(5)
    plan = tg.GroupedPlan(ROWS, N, K, EXPERTS)
    (A, B, offsets, want), (A2, B2, offsets2, want2) = _inputs(rng), _inputs(rng)
    C = torch.full((ROWS, N), float("nan"), dtype=torch.float16, device="cuda")
    side = torch.cuda.Stream()
    plan(A, B, offsets, C)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):  # the stream that the eager calls take
        plan(A, B, offsets, C)
    outs = [torch.full((ROWS, N), float("nan"), dtype=torch.float16, device="cuda")
            for _ in range(40)]
    C.fill_(float("nan"))
    torch.cuda.synchronize()
    for out in outs:
        graph.replay()
        plan(A2, B2, offsets2, out, stream=side)
    torch.cuda.synchronize()
    assert plan.device_status() == 0
    assert torch.equal(C, want)
    for out in outs:
        assert torch.equal(out, want2)


def test_a_graph_gives_its_counter_back():
    """More captured launches, one graph after the other, than there are counters."""
    import torch

    import tma_pipelined_tensor_fp16_gb300 as tg
    plan = tg.GroupedPlan(8, 8, 8, 1)
    A, B = (torch.ones(s, dtype=torch.float16, device="cuda") for s in ((8, 8), (1, 8, 8)))
    offsets = torch.tensor([0, 8], dtype=torch.int32, device="cuda")
    C = torch.zeros((8, 8), dtype=torch.float16, device="cuda")
    plan(A, B, offsets, C)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(340):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            for _ in range(200):
                plan(A, B, offsets, C)
        C.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert (C == 8).all()
        del graph
