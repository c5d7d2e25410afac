"""nvfp4 with a tensor scale of the caller's: any number from 0 to the largest, as other programs
choose it (largest / 2688), is used as it is.

With t no power of two, 6 t, s t and the quotients are each rounded to fp32: a quotient is off
by less than 2^-22 of itself, so a code or a scale is that of x or of x made larger or smaller
by that.  Powers of two lose nothing, at the ends of fp32's range neither."""
import numpy as np
import pytest

import mx_util
from expert_util import assert_within, device

pytestmark = pytest.mark.gpu

OFF = 2.0 ** -22


@pytest.fixture(scope="module", autouse=True)
def _built():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()


def _inputs(rng, rows, K):
    x = rng.standard_normal((rows, K)) * 2.0 ** rng.integers(-12, 12, (rows, 1))
    x = x.astype(np.float16)
    x[::3, :16] = 0.0
    x[1::4, 16:32] = 2.0 ** -24
    x[2::5, -1], x[3::5, 40] = 65504.0, -65504.0
    return x


def _quantized(x, t, transpose):
    """(MXTensor, scales, codes one to an entry) of x by the given scale."""
    import torch

    import tma_pipelined_tensor_fp16_gb300 as tg
    scale = torch.tensor([t], dtype=torch.float32, device="cuda")
    Q = tg.mx_quantize(device(x.T.copy() if transpose else x), "nvfp4", transpose=transpose,
                       tensor_scale=scale)
    assert Q.tensor_scale is scale
    codes, scales = [v.cpu().numpy() for v in Q.to_codes()]
    assert float(scale) == np.float32(t) or np.isnan(t)
    return Q, scales, mx_util.unpack(codes, Q.K, "nvfp4")


@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("t", ["largest", 0.3, 1.9999, 3e-3, 7.7e-7, 1e4, 1e-15])
def test_no_power_of_two(t, transpose):
    import torch

    import tma_pipelined_tensor_fp16_gb300 as tg
    rng = np.random.default_rng(7)
    x = _inputs(rng, 48, 200)
    t = float(np.float32(np.abs(x.astype(np.float64)).max() / 2688.0 if t == "largest" else t))
    Q, scales, codes = _quantized(x, t, transpose)
    kinds = [mx_util.quantize(x.astype(np.float64) * f, "nvfp4", t) for f in (1, 1 + OFF, 1 - OFF)]
    assert np.logical_or.reduce([scales == k[1] for k in kinds]).all()
    levels = mx_util.e4m3_values()
    step = np.repeat(levels[scales] * t, 16, axis=1)[:, :Q.K]
    near = [mx_util.nearest(x / step * f, mx_util.E2M1) for f in (1, 1 + OFF, 1 - OFF)]
    assert np.logical_or.reduce([(codes & 7) == n for n in near]).all()
    assert (((codes & 8) != 0) == np.signbit(x)).all()
    # the values, rounded once, and a product of them
    want = mx_util.values(codes, scales, "nvfp4", t)
    full = Q.values(torch.empty(Q.rows, Q.K, device="cuda")).cpu().numpy()
    assert np.array_equal(full, want.astype(np.float32))
    with np.errstate(over="ignore"):
        assert np.array_equal(Q.values().cpu().numpy(), full.astype(np.float16))
    C = tg.MXPlan(Q.rows, Q.rows, Q.K, format="nvfp4", out="f32")(Q, Q).cpu().numpy()
    ref, size = want @ want.T, np.abs(want) @ np.abs(want).T
    # and the product of the tensor scales, and that with the sum, each rounded
    tol = Q.K * 2.0 ** -23 * size + 2.0 ** -22 * np.abs(ref) + 2.0 ** -149
    fits = np.abs(ref) < 3e38
    assert_within(C[fits], ref[fits], tol[fits], "product")


@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("t", [0.0, 2.0 ** -149, 2.0 ** -126, 2.0 ** -120, 2.0 ** -115, 2.0 ** -101,
                               2.0 ** -100, 2.0 ** -60, 2.0 ** 60, 2.0 ** 100, 2.0 ** 101,
                               2.0 ** 126, 2.0 ** 127, 3.4e38, float("inf")])
def test_the_ends_of_the_range(t, transpose):
    """Zeros stay zeros, values beyond 2688 t are cut off at 6 * 448 * t and those far below
    t round to zero."""
    import torch
    t = float(np.float32(t))
    x = _inputs(np.random.default_rng(8), 48, 200)
    Q, scales, codes = _quantized(x, t, transpose)
    near = min(max(t, 2.0 ** -140), 2.0 ** 140)  # a limit that divides
    want_c, want_s, _ = mx_util.quantize(x.astype(np.float64), "nvfp4", near)
    assert (scales == want_s).all() and (codes == want_c).all()
    if np.isfinite(t):
        full = Q.values(torch.empty(Q.rows, Q.K, device="cuda")).cpu().numpy()
        want = mx_util.values(codes, scales, "nvfp4", t)
        assert np.array_equal(full, want.astype(np.float32))


@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("t", [-1.0, -2.0 ** -130, float("nan"), -float("inf")])
def test_no_scale_at_all(t, transpose):
    x = _inputs(np.random.default_rng(9), 16, 72)
    Q, scales, _ = _quantized(x, t, transpose)
    assert (scales == 127).all() and bool(Q.values().isnan().all())

