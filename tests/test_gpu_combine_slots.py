"""Rows in slot order back to their tokens, with dropped slots, against numpy in 64
bits."""
import numpy as np
import pytest

from expert_util import assert_same, assert_within, device, integers, normals, routing, tolerance

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()


@pytest.mark.parametrize("out", ["f16", "f32"])
@pytest.mark.parametrize("weighted", [False, True])
@pytest.mark.parametrize("tokens,topk,experts,drop,width", [
    (1, 1, 2, 0.0, 8), (3, 6, 160, 0.3, 5120), (37, 2, 5, 0.5, 72), (300, 8, 16, 0.1, 264),
    (9, 1, 4, 1.0, 2048)])
def test_dropped_slots(tokens, topk, experts, drop, width, weighted, out):
    import torch

    import tma_pipelined_tensor_fp16_gb300 as tg
    rng = np.random.default_rng(tokens + width)
    ids = routing(rng, tokens, topk, experts, drop)
    kept = (ids >= 0) & (ids < experts)
    Ys = normals(rng, (tokens, topk, width))
    w = rng.random((tokens, topk)).astype(np.float32) if weighted else \
        np.ones((tokens, topk), np.float32)
    terms = np.where(kept[:, :, None], Ys.astype(np.float64) * w[:, :, None], 0.0)
    Ys[~kept], w[~kept] = np.inf, np.nan  # neither is used
    Y = torch.full((tokens, width), float("nan"), device="cuda",
                   dtype=torch.float16 if out == "f16" else torch.float32)
    got = tg.ExpertRoute(tokens, topk, experts).combine_slots(
        device(Ys.reshape(-1, width)), Y, weights=device(w) if weighted else None, ids=device(ids))
    ref = terms.sum(1)
    assert_within(got.cpu().numpy(), ref, tolerance(ref, np.abs(terms).sum(1), topk, out))


def test_no_ids_no_drops():
    import tma_pipelined_tensor_fp16_gb300 as tg
    rng = np.random.default_rng(3)
    Ys = integers(rng, (5 * 3, 40))
    got = tg.ExpertRoute(5, 3, 8).combine_slots(device(Ys))
    assert_same(got.cpu().numpy(), Ys.astype(np.float64).reshape(5, 3, 40).sum(1), "f16")


def test_refusals():
    import torch

    import tma_pipelined_tensor_fp16_gb300 as tg
    Ys = torch.zeros((8, 64), dtype=torch.float16, device="cuda")
    route = tg.ExpertRoute(4, 2, 3)
    with pytest.raises(TypeError):
        route.combine_slots(Ys, ids=torch.zeros((4, 2), dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):
        route.combine_slots(Ys, ids=torch.zeros((8,), dtype=torch.int32, device="cuda"))
