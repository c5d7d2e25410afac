"""Plans beside another one, with its status record: for batches that change their length."""
import numpy as np
import pytest

import mx_util
from expert_util import assert_same, device

pytestmark = pytest.mark.gpu

SIZES = [(1, 264, 520), (40, 136, 1024), (700, 520, 2048)]  # rows, single CTAs or pairs


@pytest.fixture(scope="module", autouse=True)
def _built():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()


def _operands(rng, M, N, K, format):
    import tma_pipelined_tensor_fp16_gb300 as tg
    made = []
    for rows in (M, N):
        packed, scales, _, v = mx_util.random_operand(rng, rows, K, format, True)
        made.append((tg.MXTensor.from_codes(device(packed), device(scales), K, format), v))
    return made


@pytest.mark.parametrize("format", ["mxfp8", "mxfp4", "nvfp4"])
def test_products_and_the_status(format):
    import torch

    import tma_pipelined_tensor_fp16_gb300 as tg
    from tma_pipelined_tensor_fp16_gb300 import binding
    rng = np.random.default_rng(1)
    first = tg.MXPlan(8, 8, 64, format=format)
    plans = [tg.MXPlan(*s, format=format, out="f32", beside=first) for s in SIZES]
    sets = [_operands(rng, *s, format) for s in SIZES]
    for plan, ((A, a), (B, b)) in zip(plans, sets):
        assert plan.describe() == tg.MXPlan(plan.M, plan.N, plan.K, format=format,
                                            out="f32").describe()
        assert_same(plan(A, B).cpu().numpy(), a @ b.T, "f32", plan.describe())
    # a wait that runs out in one is reported by each, once
    plans[1].set_wait(100, 1)
    plans[1](sets[1][0][0], sets[1][1][0])
    torch.cuda.synchronize()
    assert first.device_status() == binding.GEMM_ERR_TIMEOUT
    assert [p.device_status() for p in plans + [first]] == [0] * 4
    plans[1].set_wait()
    # the record outlives the plan that made it
    first.close()
    for plan, ((A, a), (B, b)) in zip(plans, sets):
        assert_same(plan(A, B).cpu().numpy(), a @ b.T, "f32", plan.describe())
        assert plan.device_status() == 0
        plan.close()


def test_a_new_length_while_capturing():
    """A shared expert's step at a length that it has not seen, captured: no call waits.  Its
    replays go on when the plans have left the cache."""
    import torch

    import tma_pipelined_tensor_fp16_gb300 as tg
    from tma_pipelined_tensor_fp16_gb300 import expert_layer
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    S1, S2 = (torch.randn(s, generator=g, device="cuda").mul_(0.1).half()
              for s in ((200, 136), (136, 200)))
    shared = expert_layer.SharedExpert(S1, S2, "mxfp8")
    dS = torch.empty(200, 136, device="cuda"), torch.empty(136, 200, device="cuda")
    X = torch.randn((333, 136), generator=g, device="cuda").half()

    def step(x):
        Y, A = shared.forward(tg.mx_quantize(x))
        return (Y, A) + shared.backward(Y, A, x, dS)
    step(X[:40].contiguous())  # everything has run once, at another length
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step(X)
    for n in range(1, 40):
        step(X[:n].contiguous())
    assert shared._plan.cache_info().currsize <= 64
    graph.replay()
    got = [t.clone() for t in held]
    assert all(torch.equal(a, b) for a, b in zip(got, step(X)))
    assert shared.device_status() == 0


def test_refusals():
    import tma_pipelined_tensor_fp16_gb300 as tg
    first = tg.MXPlan(8, 8, 64, format="mxfp8")
    with pytest.raises(ValueError):
        tg.MXPlan(8, 8, 64, format="mxfp4", beside=first)
    with pytest.raises(tg.GemmError):
        tg.MXPlan(8, 12, 64, format="mxfp8", beside=first)
