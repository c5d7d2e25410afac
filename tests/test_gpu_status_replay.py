"""A timeout inside a replayed CUDA graph is reported by every replay that has one:
a barrier that nothing completes (debug_stall), bounded by wait_budget_ms."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()


def test_every_stalled_replay_is_reported():
    import torch

    import tma_pipelined_tensor_fp16_gb300 as pkg
    from tma_pipelined_tensor_fp16_gb300 import binding
    A = torch.ones((256, 128), dtype=torch.float16, device="cuda")
    C = torch.zeros((256, 256), dtype=torch.float32, device="cuda")
    plan = pkg.Plan(256, 256, 128, out="f32", variant="persistent", debug_stall=1,
                    wait_budget_ms=50)
    plan(A, A, C)
    torch.cuda.synchronize()
    assert plan.device_status() == binding.GEMM_ERR_TIMEOUT
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        plan(A, A, C)
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert plan.device_status() == binding.GEMM_ERR_TIMEOUT
        assert plan.device_status() == binding.GEMM_OK  # read and clear
    plan.close()
