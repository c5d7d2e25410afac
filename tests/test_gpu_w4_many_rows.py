"""Products with 4-bit weights for many rows, where the weights are expanded for
the GEMM: no weight is rounded, no product overflows in between, and an infinity
reaches its own row only, as with few rows."""
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


SHAPES = [(1100, 264, 64, 32), (2000, 136, 256, 32), (1500, 1032, 1152, 128),
          (3001, 72, 320, 64)]


def _codes(rng, N, K, group, scales, zeros):
    packed = rng.integers(0, 256, (N, K // 2)).astype(np.uint8)
    z = rng.integers(0, 16, scales.shape).astype(np.uint8) if zeros else None
    q = np.stack([packed & 15, packed >> 4], -1).reshape(N, K // group, group)
    w = (q.astype(np.float64) - (8.0 if z is None else z[..., None])) * \
        scales.astype(np.float64)[..., None]
    return packed, z, w.reshape(N, K)


def _plan(M, N, K, group, out, **kw):
    import tma_pipelined_tensor_fp16_gb300 as tg
    plan = tg.W4Plan(M, N, K, group=group, out=out, **kw)
    assert plan.describe().startswith("w4 expand"), plan.describe()
    return plan


def _product(plan, X, packed, scales, z):
    import torch

    import tma_pipelined_tensor_fp16_gb300 as tg
    Y = torch.full((plan.M + 1, plan.N), float("nan"), dtype=plan.dtype, device="cuda")
    plan(device(X), device(packed), device(scales), Y[:-1],
         zeros=None if z is None else device(z))
    torch.cuda.synchronize()
    assert plan.device_status() == 0, tg.gemm_last_error() + "; " + plan.describe()
    assert torch.isnan(Y[-1]).all(), "wrote past the end"
    return Y[:-1].cpu().numpy()


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("M,N,K,group", SHAPES)
def test_no_weight_is_rounded(M, N, K, group, zeros):
    """fp32 sums over the 2 K products of both parts."""
    rng = np.random.default_rng(M + K)
    scales = (rng.random((N, K // group)) + 0.5).astype(np.float16)
    packed, z, w = _codes(rng, N, K, group, scales, zeros)
    X = normals(rng, (M, K))
    got = _product(_plan(M, N, K, group, "f32"), X, packed, scales, z)
    x = X.astype(np.float64)
    assert_within(got, x @ w.T, tolerance(None, np.abs(x) @ np.abs(w).T, 2 * K, "f32"))


@pytest.mark.parametrize("out", ["f16", "f32"])
@pytest.mark.parametrize("M,N,K,group", SHAPES)
def test_weights_of_more_bits_than_a_half(M, N, K, group, out):
    """Scales of eleven bits times codes: whole numbers up to 15 * 2047 over 64, which
    fp16 does not hold.  Every sum is below 2^24 / 64, so fp32 does, in any order."""
    rng = np.random.default_rng(N + K)
    scales = (rng.integers(1024, 2048, (N, K // group)) / 64.0).astype(np.float16)
    packed, z, w = _codes(rng, N, K, group, scales, True)
    X = np.zeros((M, K), np.float16)
    for c in rng.integers(0, K, (16, M)):  # at most 16 entries of 1 a row: 16 * 15 * 2047 < 2^24
        X[np.arange(M), c] = 1.0
    got = _product(_plan(M, N, K, group, out), X, packed, scales, z)
    assert_same(got, X.astype(np.float64) @ w.T, out)


def test_weights_beyond_half_s_range():
    """A scale of 60000: the weights pass 65504, the sums stay finite in fp32."""
    rng = np.random.default_rng(3)
    M, N, K, group = 1300, 72, 192, 64
    scales = np.full((N, K // group), 2.0, np.float16)
    scales[5] = 60000.0  # every sum of that row is a multiple of 60000
    packed, z, w = _codes(rng, N, K, group, scales, True)
    assert np.abs(w).max() > 65504
    X = integers(rng, (M, K))
    plan = _plan(M, N, K, group, "f32")
    assert_same(_product(plan, X, packed, scales, z), X.astype(np.float64) @ w.T, "f32")


@pytest.mark.parametrize("value", [np.inf, -np.inf, np.nan])
def test_entry_that_is_not_finite_reaches_its_own_row_only(value):
    rng = np.random.default_rng(9)
    M, N, K, group = 1200, 48, 256, 64
    scales = (2.0 ** rng.integers(-2, 2, (N, K // group))).astype(np.float16)
    packed, z, w = _codes(rng, N, K, group, scales, False)
    plan = _plan(M, N, K, group, "f32")
    X = integers(rng, (M, K))
    want = X.astype(np.float64) @ w.T
    bad = X.copy()
    bad[700, 17] = value
    got = _product(plan, bad, packed, scales, z)
    rest = np.arange(M) != 700
    assert_same(got[rest], want[rest], "f32")
    with np.errstate(invalid="ignore"):
        assert np.array_equal(got[700], (value * w[:, 17]).astype(np.float32), equal_nan=True)
    # and nothing of it stays in the plan
    assert_same(_product(plan, X, packed, scales, z), want, "f32")


def test_graph_follows_the_inputs():
    """A replay takes the form that its inputs need."""
    import torch
    rng = np.random.default_rng(21)
    M, N, K, group = 1100, 64, 256, 64
    scales = np.full((N, K // group), 0.5, np.float16)
    packed, z, w = _codes(rng, N, K, group, scales, True)
    X = integers(rng, (M, K))
    want = X.astype(np.float64) @ w.T
    plan = _plan(M, N, K, group, "f16")
    dX, dP, dS, dZ = device(X), device(packed), device(scales), device(z)
    Y = torch.empty((M, N), dtype=torch.float16, device="cuda")
    plan(dX, dP, dS, Y, zeros=dZ)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        plan(dX, dP, dS, Y, zeros=dZ)
    for value in (1.0, np.inf, 2.0):
        X[3, 5] = value
        dX[3, 5] = float(value)
        Y.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        got = Y.cpu().numpy()
        rest = np.arange(M) != 3
        assert_same(got[rest], want[rest], "f16")
        if np.isfinite(value):
            assert_same(got[3], X[3].astype(np.float64) @ w.T, "f16")
        else:
            assert not np.isfinite(got[3][w[:, 5] != 0]).any()
    assert plan.device_status() == 0


@pytest.mark.parametrize("M,N,K,group", SHAPES[1:3])
def test_rounded_weights_on_request(M, N, K, group):
    """Half a unit in the last place of each weight; exact where a weight is fp16."""
    rng = np.random.default_rng(M)
    for exact in (True, False):
        scales = (2.0 ** rng.integers(-2, 2, (N, K // group)) if exact else
                  rng.random((N, K // group)) + 0.5).astype(np.float16)
        packed, z, w = _codes(rng, N, K, group, scales, True)
        X = integers(rng, (M, K)) if exact else normals(rng, (M, K))
        plan = _plan(M, N, K, group, "f32", weights="rounded")
        assert "weights=rounded" in plan.describe()
        got = _product(plan, X, packed, scales, z)
        x = X.astype(np.float64)
        mag = np.abs(x) @ np.abs(w).T
        if exact:
            assert_same(got, x @ w.T, "f32")
        else:
            assert_within(got, x @ w.T, tolerance(None, mag, K, "f32") + 2.0 ** -11 * mag)


@pytest.mark.parametrize("M,N,K,group", [(1100, 136, 4096, 64), (2000, 264, 8192, 128),
                                         (70, 4096, 8192, 32)])
def test_long_sums_in_fp32(M, N, K, group):
    """With fp32 outputs many rows are as exact as few ones: each group's sum is whole
    q - zero times fp16, and the K / group of them are added in fp32 with rounding to
    nearest, 2^-24 each, so the error stays below 8 * 2^-23 of the result's norm."""
    import torch

    import tma_pipelined_tensor_fp16_gb300 as tg
    rng = np.random.default_rng(K)
    scales = (rng.random((N, K // group)) + 0.5).astype(np.float16)
    packed, z, w = _codes(rng, N, K, group, scales, True)
    X = normals(rng, (M, K))
    plan = tg.W4Plan(M, N, K, group=group, out="f32")
    got = _product(plan, X, packed, scales, z).astype(np.float64)
    want = (torch.from_numpy(X).cuda().double() @ torch.from_numpy(w).cuda().t()).cpu().numpy()
    assert np.linalg.norm(got - want) < 8 * 2.0 ** -23 * np.linalg.norm(want), plan.describe()
