"""Products with 4-bit weights against numpy in 64 bits: whole-number rows with
power-of-two scales bit for bit, random ones within the tolerance of
expert_util (plus the stated rounding of the weights to fp16 above 64 rows)."""
import numpy as np
import pytest

from expert_util import assert_same, assert_within, device, integers, normals, tolerance

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()


def _weights(rng, lead, N, K, group, zeros, exact):
    packed = rng.integers(0, 256, lead + (N, K // 2)).astype(np.uint8)
    shape = lead + (N, K // group)
    if exact:
        scales = (2.0 ** rng.integers(-2, 2, shape)).astype(np.float16)
    else:
        scales = (rng.random(shape) + 0.5).astype(np.float16)
    z = rng.integers(0, 16, shape).astype(np.uint8) if zeros else None
    q = np.stack([packed & 15, packed >> 4], -1).reshape(lead + (N, K // group, group))
    w = (q.astype(np.float64) - (8.0 if z is None else z[..., None])) * scales[..., None]
    return packed, scales, z, w.reshape(lead + (N, K))


def _run(M, N, K, group, zeros, out, exact, rng):
    import torch

    import tma_pipelined_tensor_fp16_gb300 as tg
    packed, scales, z, w = _weights(rng, (), N, K, group, zeros, exact)
    X = integers(rng, (M, K)) if exact else normals(rng, (M, K))
    plan = tg.W4Plan(M, N, K, group=group, out=out)
    Y = torch.full((M + 1, N), float("nan"), dtype=plan.dtype, device="cuda")
    plan(device(X), device(packed), device(scales), Y[:-1],
         zeros=device(z) if zeros else None)
    torch.cuda.synchronize()
    assert plan.device_status() == 0, tg.gemm_last_error() + "; " + plan.describe()
    assert torch.isnan(Y[-1]).all(), "wrote past the end"
    X = X.astype(np.float64)
    return Y[:-1].cpu().numpy(), X @ w.T, np.abs(X) @ np.abs(w).T, plan.describe()


SHAPES = [  # M, N, K, group
    (1, 8, 32, 32), (1, 8, 128, 128), (1, 16, 64, 64), (2, 24, 96, 32), (1, 4096, 2048, 128),
    (3, 40, 352, 32), (7, 1000, 4160, 64), (8, 264, 2688, 128), (9, 72, 1056, 32),
    (16, 520, 1152, 128), (17, 136, 320, 64), (33, 200, 2336, 32), (63, 120, 640, 128),
    (64, 72, 1088, 64), (1, 128, 16384, 128), (5, 32, 8192, 32),
]


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("out", ["f16", "f32"])
@pytest.mark.parametrize("M,N,K,group", SHAPES)
def test_integers_exact(M, N, K, group, out, zeros):
    rng = np.random.default_rng(M * 1000 + N + K)
    got, want, _, what = _run(M, N, K, group, zeros, out, True, rng)
    assert_same(got, want, out, what)


@pytest.mark.parametrize("M,N,K,group", SHAPES)
def test_random(M, N, K, group):
    rng = np.random.default_rng(M + N + K)
    for out in ("f16", "f32"):
        got, want, mag, what = _run(M, N, K, group, True, out, False, rng)
        assert_within(got, want, tolerance(want, mag, K, out), what)


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("M,N,K,group", [(65, 72, 96, 32), (300, 264, 640, 128),
                                         (1000, 520, 1088, 64)])
def test_many_rows(M, N, K, group, zeros):
    """Above 64 rows: exact where the weights are fp16 numbers, else within
    half a unit in the last place of each weight."""
    rng = np.random.default_rng(M)
    for out in ("f16", "f32"):
        got, want, _, what = _run(M, N, K, group, zeros, out, True, rng)
        assert_same(got, want, out, what)
        got, want, mag, what = _run(M, N, K, group, zeros, out, False, rng)
        assert_within(got, want, tolerance(want, mag, K, out) + 2.0 ** -11 * mag, what)


# Blocks of 64 rows: the last one of one row, half and whole, a length that ends in half
# a stage and in a part of a block, with the length on one CTA and on several.
BLOCKS = [(65, 264, 2176, 32), (128, 1032, 2112, 64), (193, 136, 4224, 128),
          (256, 520, 2208, 32), (400, 72, 4096, 64), (130, 4096, 1024, 128)]


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("M,N,K,group", BLOCKS)
def test_blocks_of_rows(M, N, K, group, zeros):
    """More rows than a block without rounding the weights."""
    rng = np.random.default_rng(M + N)
    for out in ("f16", "f32"):
        got, want, _, what = _run(M, N, K, group, zeros, out, True, rng)
        assert what.startswith("w4 rows"), what
        assert_same(got, want, out, what)
        got, want, mag, what = _run(M, N, K, group, zeros, out, False, rng)
        assert_within(got, want, tolerance(want, mag, K, out), what)


@pytest.mark.parametrize("M,N,K,group", [(2000, 136, 256, 32), (3000, 512, 512, 64),
                                         (1500, 1032, 1152, 128)])
def test_expanded(M, N, K, group):
    """Many rows take the expansion to fp16."""
    rng = np.random.default_rng(M + K)
    for zeros in (False, True):
        got, want, _, what = _run(M, N, K, group, zeros, "f32", True, rng)
        assert what.startswith("w4 expand"), what
        assert_same(got, want, "f32", what)
        got, want, mag, what = _run(M, N, K, group, zeros, "f16", False, rng)
        assert_within(got, want, tolerance(want, mag, K, "f16") + 2.0 ** -11 * mag, what)


def test_zero_points_beyond_four_bits():
    """Zero points are whole numbers 0..255 and stay exact."""
    import tma_pipelined_tensor_fp16_gb300 as tg
    rng = np.random.default_rng(8)
    packed, scales, z, _ = _weights(rng, (), 16, 64, 32, True, True)
    z = rng.integers(0, 256, z.shape).astype(np.uint8)
    q = np.stack([packed & 15, packed >> 4], -1).reshape(16, 2, 32).astype(np.float64)
    w = ((q - z[..., None]) * scales[..., None]).reshape(16, 64)
    X = integers(rng, (1, 64))
    got = tg.W4Plan(1, 16, 64, group=32, out="f32")(device(X), device(packed), device(scales),
                                                  zeros=device(z))
    assert_same(got.cpu().numpy(), X.astype(np.float64) @ w.T, "f32")


def test_infinite_entry_reaches_its_own_row_only():
    import tma_pipelined_tensor_fp16_gb300 as tg
    rng = np.random.default_rng(9)
    packed, scales, _, w = _weights(rng, (), 48, 256, 64, False, True)
    X = integers(rng, (4, 256))
    want = X.astype(np.float64) @ w.T
    X[2, 17] = np.inf
    got = tg.W4Plan(4, 48, 256, group=64, out="f32")(device(X), device(packed), device(scales))
    got = got.cpu().numpy()
    assert_same(got[[0, 1, 3]], want[[0, 1, 3]], "f32")
    sign = w[:, 17]
    assert np.array_equal(got[2][sign > 0], np.full((sign > 0).sum(), np.inf))
    assert np.array_equal(got[2][sign < 0], np.full((sign < 0).sum(), -np.inf))
    assert np.isnan(got[2][sign == 0]).all()


@pytest.mark.parametrize("tokens,topk,experts,N,K,group,drop", [
    (1, 1, 1, 16, 64, 32, 0.0), (4, 8, 64, 264, 1024, 128, 0.0), (16, 6, 8, 72, 352, 32, 0.2),
    (1, 8, 8, 40, 4096, 64, 0.0), (100, 3, 4, 24, 128, 64, 0.1), (3, 2, 300, 136, 256, 128, 0.5),
])
def test_by_expert(tokens, topk, experts, N, K, group, drop):
    """Rows of one expert together (more than a pass holds, too), dropped rows
    zero; a second product on the first one's rows (share = 1)."""
    import torch

    import tma_pipelined_tensor_fp16_gb300 as tg
    from expert_util import routing
    rng = np.random.default_rng(tokens + N)
    ids = routing(rng, tokens, topk, experts, drop)
    packed, scales, z, w = _weights(rng, (experts,), N, K, group, True, True)
    X = integers(rng, (tokens, K))
    M = tokens * topk
    for share, x in ((topk, X), (1, np.repeat(X, topk, axis=0))):
        plan = tg.W4Plan(M, N, K, group=group, out="f32", experts=experts, share=share)
        Y = torch.full((M + 1, N), float("nan"), dtype=torch.float32, device="cuda")
        plan(device(x), device(packed), device(scales), Y[:-1], zeros=device(z), ids=device(ids))
        want = np.zeros((M, N))
        for s, e in enumerate(ids.reshape(-1)):
            if 0 <= e < experts:
                want[s] = w[e] @ X[s // topk].astype(np.float64)
        assert_same(Y[:-1].cpu().numpy(), want, "f32", plan.describe())
        assert torch.isnan(Y[-1]).all()


def test_pack():
    import torch

    import tma_pipelined_tensor_fp16_gb300 as tg
    torch.manual_seed(0)
    W = torch.randn(64, 512, device="cuda")
    X = torch.randn(3, 512, device="cuda", dtype=torch.float16)
    for zeros in (False, True):
        packed, scales, z = tg.w4_pack(W, 64, zeros)
        got = tg.W4Plan(3, 64, 512, group=64, out="f32")(X, packed, scales, zeros=z)
        q = torch.stack([packed & 15, packed >> 4], -1).reshape(64, 8, 64).double()
        w = ((q - (8.0 if z is None else z[..., None].double())) * scales[..., None].double())
        # a code is at most half a step off, plus a step at a rounded zero point
        step = scales[..., None].double() * (0.51 if z is None else 1.02)
        assert ((w - W.double().reshape(64, 8, 64)).abs() <= step + 1e-6).all()
        ref = X.double() @ w.reshape(64, 512).t()
        assert (got.double() - ref).abs().max() < 1e-3


def test_stream_and_graph():
    import torch

    import tma_pipelined_tensor_fp16_gb300 as tg
    rng = np.random.default_rng(21)
    for M in (2, 100):
        packed, scales, _, w = _weights(rng, (), 64, 256, 64, False, True)
        X = integers(rng, (M, 256))
        dX, dP, dS = device(X), device(packed), device(scales)
        plan = tg.W4Plan(M, 64, 256, group=64)
        Y = torch.empty((M, 64), dtype=torch.float16, device="cuda")
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        plan(dX, dP, dS, Y, stream=s)
        s.synchronize()
        want = X.astype(np.float64) @ w.T
        assert_same(Y.cpu().numpy(), want, "f16")
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            plan(dX, dP, dS, Y)
        dX.neg_()
        graph.replay()
        torch.cuda.synchronize()
        assert_same(Y.cpu().numpy(), -want, "f16")


def test_refusals():
    import torch

    import tma_pipelined_tensor_fp16_gb300 as tg
    with pytest.raises(tg.GemmError, match="group must be"):
        tg.W4Plan(1, 64, 256, group=48)
    with pytest.raises(tg.GemmError, match="multiple of group"):
        tg.W4Plan(1, 64, 192, group=128)
    with pytest.raises(tg.GemmError, match="16 bytes"):
        tg.W4Plan(1, 60, 128)
    with pytest.raises(tg.GemmError, match="at most 1024"):
        tg.W4Plan(1025, 64, 128, experts=4)
    plan = tg.W4Plan(1, 64, 128)
    z = lambda s, d=torch.float16: torch.zeros(s, dtype=d, device="cuda")
    x, packed, scales = z((1, 128)), z((64, 64), torch.uint8), z((64, 1))
    with pytest.raises(TypeError):
        plan(x.float(), packed, scales)
    with pytest.raises(ValueError):
        plan(x, packed[:, :32].contiguous(), scales)
    with pytest.raises(ValueError, match="exactly when"):
        plan(x, packed, scales, ids=z((1,), torch.int32))
