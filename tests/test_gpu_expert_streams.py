"""A call on another stream without an output tensor: its memory may have been freed
on the current stream while work there still reads it."""
import numpy as np
import pytest

from expert_util import assert_same, device, integers, offsets_of, routing, sort_reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()


def _beside_a_late_reader(shape, dtype, call):
    """call(stream) on a stream of its own, while a copy on the current stream, queued
    behind some milliseconds of waiting, has yet to read a tensor of the given shape
    that is already freed.  Returns (result, whether the copy saw the tensor's values)."""
    import torch
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    old = torch.full(shape, 7, dtype=dtype, device="cuda")
    seen = torch.empty(shape, dtype=dtype, device="cuda")
    side.wait_stream(torch.cuda.current_stream())
    torch.cuda._sleep(20_000_000)
    seen.copy_(old)
    del old
    got = call(side)
    side.synchronize()
    torch.cuda.synchronize()
    return got, bool((seen == 7).all())


def test_sort_and_gather():
    import torch

    import tma_pipelined_tensor_fp16_gb300 as tg
    rng = np.random.default_rng(1)
    ids = routing(rng, 700, 3, 9, 0.1)
    offsets, order, position = sort_reference(ids, 9)
    dids = device(ids)
    route, intact = _beside_a_late_reader(
        (2100,), torch.int32, lambda s: tg.ExpertRoute(700, 3, 9).sort(dids, stream=s))
    assert intact
    assert (route.order.cpu().numpy() == order).all()
    assert (route.position.cpu().numpy() == position).all()
    X = integers(rng, (700, 128))
    dX = device(X)
    Xs, intact = _beside_a_late_reader((2100, 128), torch.float16,
                                       lambda s: route.gather(dX, stream=s))
    assert intact
    keep = offsets[-1]
    assert_same(Xs.cpu().numpy()[:keep], X[order[:keep] // 3], "f16")


def test_plans():
    import torch

    import tma_pipelined_tensor_fp16_gb300 as tg
    rng = np.random.default_rng(2)
    A, B = integers(rng, (300, 64)), integers(rng, (2, 256, 64))
    dA, dB, offs = device(A), device(B), device(offsets_of([100, 200]))
    grouped = tg.GroupedPlan(300, 256, 64, 2)
    C, intact = _beside_a_late_reader((300, 256), torch.float16,
                                      lambda s: grouped(dA, dB, offs, stream=s))
    assert intact
    want = np.concatenate([A[:100].astype(float) @ B[0].T, A[100:].astype(float) @ B[1].T])
    assert_same(C.cpu().numpy(), want, "f16")
    packed = rng.integers(0, 256, (512, 32)).astype(np.uint8)
    q = np.stack([packed & 15, packed >> 4], -1).reshape(512, 64).astype(float) - 8
    scales = torch.ones((512, 1), dtype=torch.float16, device="cuda")
    dP, x = device(packed), device(A[:4])
    w4 = tg.W4Plan(4, 512, 64, group=64)
    Y, intact = _beside_a_late_reader((4, 512), torch.float16,
                                      lambda s: w4(x, dP, scales, stream=s))
    assert intact
    assert_same(Y.cpu().numpy(), A[:4].astype(float) @ q.T, "f16")


def test_capture_beside_the_sort_s_stream():
    """Tables made on one stream and used in a graph, which captures on another."""
    import torch

    import tma_pipelined_tensor_fp16_gb300 as tg
    rng = np.random.default_rng(3)
    ids = routing(rng, 60, 2, 5, 0.0)
    X = integers(rng, (60, 64))
    route = tg.ExpertRoute(60, 2, 5).sort(device(ids))
    dX = device(X)
    Xs = torch.empty((120, 64), dtype=torch.float16, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        route.gather(dX, Xs)
    graph.replay()
    torch.cuda.synchronize()
    assert_same(Xs.cpu().numpy(), X[sort_reference(ids, 5)[1] // 2], "f16")
    del route, graph
    torch.cuda.synchronize()
    torch.zeros(1000, device="cuda").sum().item()
