"""Offsets that no sort writes: a table that descends gives zeros, one that leaves
[0, rows] is taken as far as it goes.  Every access stays inside the tensors."""
import numpy as np
import pytest

from expert_util import assert_same, device, integers

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()


@pytest.mark.parametrize("tile", ["128x128", "128x256", "256x256"])
@pytest.mark.parametrize("op", ["forward", "grad_input"])
@pytest.mark.parametrize("experts,table", [
    (3, [0, 300, 200, 500]), (150, [0, 700] * 75 + [0]), (1, [5, 3])])
def test_descending(op, tile, experts, table):
    import torch

    import tma_pipelined_tensor_fp16_gb300 as tg
    rows, N, K = 700, 136, 72
    plan = tg.GroupedPlan(rows, N, K, experts, op=op, tile=tile)
    sp, sq, so = plan.shapes()
    out = torch.full((so[0] + 1, so[1]), float("nan"), dtype=torch.float16, device="cuda")
    plan(torch.ones(sp, dtype=torch.float16, device="cuda"),
         torch.ones(sq, dtype=torch.float16, device="cuda"),
         torch.tensor(table, dtype=torch.int32, device="cuda"), out[:-1])
    torch.cuda.synchronize()
    assert plan.device_status() == 0
    assert (out[:-1] == 0).all() and torch.isnan(out[-1]).all()


@pytest.mark.parametrize("tile", ["128x128", "256x256"])
def test_past_the_ends(tile):
    """The first expert from a negative row on, the last one past the rows."""
    import tma_pipelined_tensor_fp16_gb300 as tg
    rng = np.random.default_rng(1)
    A, B = integers(rng, (300, 64)), integers(rng, (3, 136, 64))
    plan = tg.GroupedPlan(300, 136, 64, 3, out="f32", tile=tile)
    got = plan(device(A), device(B), device(np.array([-7, 100, 150, 2 ** 31 - 1], np.int32)))
    want = np.concatenate([A[a:b].astype(np.float64) @ B[e].astype(np.float64).T
                           for e, (a, b) in enumerate([(0, 100), (100, 150), (150, 300)])])
    assert_same(got.cpu().numpy(), want, "f32")
