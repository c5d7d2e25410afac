"""Waits that run out inside the grouped and the 4-bit kernels: a role first waits on a
barrier that nothing completes (no fault, no trap: a flag nobody sets), with copies and
MMAs of other roles under way.  The run ends in bounded time with GEMM_ERR_TIMEOUT, and
the plan's next run is right."""
import time

import numpy as np
import pytest

from expert_util import assert_same, device, integers, offsets_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()


def _stalled(plan, run, stall):
    import torch

    import tma_pipelined_tensor_fp16_gb300 as tg
    from tma_pipelined_tensor_fp16_gb300 import binding
    plan.set_wait(100, stall)
    t0 = time.time()
    run()
    torch.cuda.synchronize()
    assert time.time() - t0 < 10.0
    assert plan.device_status() == binding.GEMM_ERR_TIMEOUT
    assert "timed out" in tg.gemm_last_error()
    assert plan.device_status() == binding.GEMM_OK
    plan.set_wait()


@pytest.mark.parametrize("stall", [1, 2])
@pytest.mark.parametrize("tile", ["128x128", "128x256", "256x256"])
@pytest.mark.parametrize("op", ["forward", "grad_input", "grad_weight"])
def test_grouped(op, tile, stall):
    import torch

    import tma_pipelined_tensor_fp16_gb300 as tg
    rng = np.random.default_rng(3)
    counts = [700, 33, 0, 515, 90]
    offsets = offsets_of(counts)
    rows, N, K = sum(counts), 1032, 520
    plan = tg.GroupedPlan(rows, N, K, len(counts), op=op, out="f32", tile=tile)
    sp, sq, so = plan.shapes()
    P, Q = integers(rng, sp), integers(rng, sq)
    dP, dQ, dO = device(P), device(Q), device(offsets)
    C = torch.empty(so, dtype=torch.float32, device="cuda")
    _stalled(plan, lambda: plan(dP, dQ, dO, C), stall)
    want = np.zeros(so)
    P, Q = P.astype(np.float64), Q.astype(np.float64)
    for e in range(len(counts)):
        s = slice(offsets[e], offsets[e + 1])
        if op == "forward":
            want[s] = P[s] @ Q[e].T
        elif op == "grad_input":
            want[s] = P[s] @ Q[e]
        else:
            want[e] = P[s].T @ Q[s]
    for _ in range(2):
        C.fill_(float("nan"))
        plan(dP, dQ, dO, C)
        torch.cuda.synchronize()
        assert plan.device_status() == 0
        assert_same(C.cpu().numpy(), want, "f32", plan.describe())


@pytest.mark.parametrize("stall", [1, 2])
@pytest.mark.parametrize("M,N,K,group,experts", [
    (1, 4096, 4096, 128, 0), (9, 264, 8192, 32, 0), (20, 520, 2048, 64, 0), (64, 1032, 4224, 32, 0),
    (130, 264, 2176, 128, 0), (6, 136, 4096, 64, 3)])
def test_w4(M, N, K, group, experts, stall):
    import torch

    import tma_pipelined_tensor_fp16_gb300 as tg
    rng = np.random.default_rng(5)
    lead = (experts,) if experts else ()
    packed = rng.integers(0, 256, lead + (N, K // 2)).astype(np.uint8)
    q = np.stack([packed & 15, packed >> 4], -1).reshape(lead + (N, K)).astype(np.float64) - 8
    X = integers(rng, (M, K))
    plan = tg.W4Plan(M, N, K, group=group, out="f32", experts=experts)
    assert plan.describe().startswith("w4 rows")
    scales = torch.ones(lead + (N, K // group), dtype=torch.float16, device="cuda")
    ids = rng.integers(0, experts, M).astype(np.int32) if experts else None
    dX, dP, dI = device(X), device(packed), None if ids is None else device(ids)
    Y = torch.empty((M, N), dtype=torch.float32, device="cuda")
    _stalled(plan, lambda: plan(dX, dP, scales, Y, ids=dI), stall)
    x = X.astype(np.float64)
    want = x @ q.T if not experts else np.stack([q[e] @ x[m] for m, e in enumerate(ids)])
    for _ in range(2):
        Y.fill_(float("nan"))
        plan(dX, dP, scales, Y, ids=dI)
        torch.cuda.synchronize()
        assert plan.device_status() == 0
        assert_same(Y.cpu().numpy(), want, "f32", plan.describe())


def test_refusals():
    import tma_pipelined_tensor_fp16_gb300 as tg
    plan = tg.GroupedPlan(8, 8, 8, 1)
    for budget, stall in ((-1, 0), (0, 3), (0, -1)):
        with pytest.raises(tg.GemmError):
            plan.set_wait(budget, stall)
