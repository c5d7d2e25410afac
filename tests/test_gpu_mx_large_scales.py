"""Values of nvfp4 matrices whose tensor scale is large: s t beyond fp32, q s t within it."""
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



@pytest.mark.parametrize("K", [200, 203])
def test_values_of_large_scales(K):
    import torch

    import tma_pipelined_tensor_fp16_gb300 as tg
    rng = np.random.default_rng(K)
    codes = rng.integers(0, 16, (40, K)).astype(np.uint8)
    scales = rng.integers(1, 127, (40, -(-K // 16))).astype(np.uint8)
    t = 2.0 ** 120
    scale = torch.tensor([t], device="cuda")
    Q = tg.MXTensor.from_codes(device(mx_util.pack(codes, "nvfp4")), device(scales), K, "nvfp4",
                               scale)
    full = Q.values(torch.empty(40, K, device="cuda")).cpu().numpy()
    with np.errstate(over="ignore"):
        want = mx_util.values(codes, scales, "nvfp4", t).astype(np.float32)
        assert np.isinf(want).any() and (want == 0).any()
        assert np.array_equal(full, want)
        assert np.array_equal(Q.values().cpu().numpy(), want.astype(np.float16))
