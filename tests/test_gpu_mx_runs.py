"""Block-scaled products and the layer's operators as programs run them: overlapping runs
of one plan, graphs, other streams, waits that run out, values that are not finite."""
import time

import numpy as np
import pytest

import mx_util
from expert_util import assert_same, device

pytestmark = pytest.mark.gpu

FORMATS = ["mxfp8", "mxfp4", "nvfp4"]
CASES = [  # M, N, K, options
    (5, 520, 4096, {"kernel": "single", "split": 4}), (1, 264, 1024, {}),
    (200, 264, 2048, {"kernel": "single", "split": 2}), (1000, 1032, 1600, {"kernel": "pair"})]


@pytest.fixture(scope="module", autouse=True)
def _built():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()


def _operand(rng, rows, K, format):
    import tma_pipelined_tensor_fp16_gb300 as tg
    packed, scales, _, v = mx_util.random_operand(rng, rows, K, format, True)
    return tg.MXTensor.from_codes(device(packed), device(scales), K, format), v


@pytest.mark.parametrize("stall", [1, 2])
@pytest.mark.parametrize("format", FORMATS)
@pytest.mark.parametrize("M,N,K,options", CASES)
def test_a_wait_that_runs_out(M, N, K, options, format, stall):
    """A role first waits on a barrier that nothing completes, with the others under way: the
    run ends in bounded time with a status, and the plan's next run is right."""
    import torch

    import tma_pipelined_tensor_fp16_gb300 as tg
    from tma_pipelined_tensor_fp16_gb300 import binding
    rng = np.random.default_rng(M)
    (A, a), (B, b) = _operand(rng, M, K, format), _operand(rng, N, K, format)
    plan = tg.MXPlan(M, N, K, format=format, out="f32", **options)
    C = torch.empty((M, N), device="cuda")
    plan.set_wait(100, stall)
    t0 = time.time()
    plan(A, B, C)
    torch.cuda.synchronize()
    assert time.time() - t0 < 10.0
    assert plan.device_status() == binding.GEMM_ERR_TIMEOUT
    assert "timed out" in tg.gemm_last_error()
    assert plan.device_status() == binding.GEMM_OK
    plan.set_wait()
    for _ in range(2):
        C.fill_(float("nan"))
        plan(A, B, C)
        torch.cuda.synchronize()
        assert plan.device_status() == 0
        assert_same(C.cpu().numpy(), a @ b.T, "f32", plan.describe())


@pytest.mark.parametrize("format", FORMATS)
@pytest.mark.parametrize("M,N,K,options", CASES)
def test_overlapping_runs_and_graphs_of_one_plan(M, N, K, options, format):
    import torch

    import tma_pipelined_tensor_fp16_gb300 as tg
    rng = np.random.default_rng(M + 1)
    plan = tg.MXPlan(M, N, K, format=format, **options)
    sets = [(_operand(rng, M, K, format), _operand(rng, N, K, format)) for _ in range(4)]
    want = [a @ b.T for (_, a), (_, b) in sets]
    out = [torch.full((M, N), float("nan"), dtype=torch.float16, device="cuda") for _ in sets]
    graphs = []
    for ((A, _), (B, _)), C in list(zip(sets, out))[:2]:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            plan(A, B, C)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(5):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        for ((A, _), (B, _)), C, s in list(zip(sets, out, streams))[2:]:
            plan(A, B, C, stream=s)
    torch.cuda.synchronize()
    assert plan.device_status() == 0
    for C, w in zip(out, want):
        assert_same(C.cpu().numpy(), w, "f16", plan.describe())


@pytest.mark.parametrize("format", FORMATS)
@pytest.mark.parametrize("M,N,K,options", CASES)
def test_rows_that_are_not_finite_stay_alone(M, N, K, options, format):
    """A NaN scale makes its row (of A) or column (of B) NaN and no other."""
    import torch

    import tma_pipelined_tensor_fp16_gb300 as tg
    rng = np.random.default_rng(M + 2)
    x = rng.standard_normal((M, K)).astype(np.float16)
    w = rng.standard_normal((N, K)).astype(np.float16)
    plan = tg.MXPlan(M, N, K, format=format, out="f32", **options)
    clean = plan(tg.mx_quantize(device(x), format), tg.mx_quantize(device(w), format))
    x[M // 2, 77] = np.inf
    w[N - 3, 5] = np.nan
    # nvfp4's tensor scale does not count them, but they were the largest of nothing here
    got = plan(tg.mx_quantize(device(x), format), tg.mx_quantize(device(w), format))
    torch.cuda.synchronize()
    got, clean = got.cpu().numpy(), clean.cpu().numpy()
    assert np.isnan(got[M // 2]).all() and np.isnan(got[:, N - 3]).all()
    keep = np.ones((M, N), bool)
    keep[M // 2] = keep[:, N - 3] = False
    assert np.isfinite(got[keep]).all()
    if format != "nvfp4":  # there the replaced values may have set the tensor scale
        assert np.array_equal(got[keep], clean[keep])


def test_operands_by_other_streams_memory():
    """Everything on a stream of the caller's, whose memory the results are."""
    import torch

    import tma_pipelined_tensor_fp16_gb300 as tg
    rng = np.random.default_rng(3)
    x = rng.standard_normal((40, 512)).astype(np.float16)
    w = rng.standard_normal((256, 512)).astype(np.float16)
    X, W, n = device(x), device(w), device(np.ones(512, np.float16))
    want = []
    for format in FORMATS:
        Z, _, Q = tg.rms_norm(X, n, residual=X, format=format)
        plan = tg.MXPlan(40, 256, 512, format=format)
        want.append((plan, plan(Q, tg.mx_quantize(W, format)), tg.rms_norm_grad(Z, X, n)))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = []
    for format, (plan, _, _) in zip(FORMATS, want):
        Z, _, Q = tg.rms_norm(X, n, residual=X, format=format, stream=s)
        Wq = tg.mx_quantize(W, format, stream=s)
        got.append((plan(Q, Wq, stream=s), tg.rms_norm_grad(Z, X, n, stream=s)))
    torch.cuda.current_stream().wait_stream(s)
    for (_, C, (dX, dw)), (D, (eX, ew)) in zip(want, got):
        assert torch.equal(C, D) and torch.equal(dX, eX) and torch.equal(dw, ew)


def test_refusals():
    import torch

    import tma_pipelined_tensor_fp16_gb300 as tg
    x = torch.zeros(8, 64, dtype=torch.float16, device="cuda")
    Q, P = tg.mx_quantize(x, "mxfp8"), tg.mx_quantize(x, "mxfp4")
    plan = tg.MXPlan(8, 8, 64, format="mxfp8")
    with pytest.raises(ValueError):
        plan(Q, P)
    with pytest.raises(ValueError):
        plan(Q, tg.mx_quantize(x[:4].contiguous(), "mxfp8"))
    with pytest.raises(TypeError):
        plan(x, Q)
    with pytest.raises(ValueError):
        plan(Q, Q, torch.empty(8, 9, dtype=torch.float16, device="cuda"))
    with pytest.raises(ValueError):
        tg.mx_quantize(x, "mxfp8", tensor_scale=torch.ones(1, device="cuda"))
    with pytest.raises(ValueError):
        tg.mx_quantize(x.t(), "mxfp8")
    with pytest.raises(tg.GemmError):
        tg.mx_quantize(torch.zeros(8, 60, dtype=torch.float16, device="cuda"), "mxfp8")
    with pytest.raises(ValueError):
        tg.mx_quantize(x, "mxfp8", out=P)
    with pytest.raises(TypeError):
        tg.mx_quantize(x.float(), "mxfp8")
    w = torch.ones(64, dtype=torch.float16, device="cuda")
    with pytest.raises(ValueError):
        tg.rms_norm(x, w, half=False)
    with pytest.raises(ValueError):
        tg.rms_norm(x, w, total=x)
    with pytest.raises(ValueError):
        tg.rms_norm(x, w[:32])
    with pytest.raises(tg.GemmError):
        tg.rms_norm(x, w, eps=-1.0)
    with pytest.raises(tg.GemmError):
        tg.rms_norm(torch.zeros(4, 12, dtype=torch.float16, device="cuda"),
                    torch.ones(12, dtype=torch.float16, device="cuda"))
    with pytest.raises(ValueError):
        tg.rms_norm_grad(x, x[:4].contiguous(), w)
    for budget, stall in ((-1, 0), (0, 3)):
        with pytest.raises(tg.GemmError):
            plan.set_wait(budget, stall)
