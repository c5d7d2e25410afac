"""The first run of a new GradClip on a stream that waits for nothing: the table of addresses
is on the device when the constructor returns."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()


@pytest.mark.parametrize("tensors", [1, 40, 3000])
def test_first_run_on_a_side_stream(tensors):
    import torch

    import tma_pipelined_tensor_fp16_gb300 as tg
    side = torch.cuda.Stream()
    grads = [torch.full((i % 300 + 1,), 2.0, device="cuda") for i in range(tensors)]
    n = sum(g.numel() for g in grads)
    torch.cuda.synchronize()
    for turn in range(20):
        with torch.cuda.stream(side):
            norm = tg.GradClip(grads, out=[torch.empty_like(g) for g in grads])(1.0)
        side.synchronize()
        assert abs(float(norm) - 2.0 * n ** 0.5) <= 1e-6 * float(norm), turn
