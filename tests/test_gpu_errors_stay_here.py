"""An error that a library call has reported is not reported again by torch's next
launch, which looks at the runtime's last error."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()


def test_out_of_memory():
    """A workspace of 4 TB: the allocation fails, nothing is launched."""
    import torch

    import tma_pipelined_tensor_fp16_gb300 as tg
    x = torch.zeros(1000, device="cuda")
    with pytest.raises(tg.GemmError, match="MemoryAllocation"):
        tg.W4Plan(4096, 1 << 25, 1 << 15, group=32)
    x += 1
    torch.cuda.synchronize()
    assert (x == 1).all()
