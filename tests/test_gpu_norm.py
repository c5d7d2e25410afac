"""The root-mean-square norm with residual and quantised rows, and its gradient, against
numpy in 64 bits.

Tolerance of z = h * rstd * w: the mean of n squares is off by at most (8 + sqrt(n)) *
2^-23 of itself (sums as in expert_util), rstd by half of that and 2^-23 for the square
root and the quotient, and the two products add 2^-23: so z by (6 + sqrt(n) / 2) * 2^-23 of
itself, plus half a unit of fp16.
"""
import numpy as np
import pytest

import mx_util
from expert_util import assert_within, device, tolerance

pytestmark = pytest.mark.gpu

FORMATS = [None, "mxfp8", "mxfp4", "nvfp4"]
SHAPES = [(1, 8), (3, 72), (16, 256), (9, 264), (17, 512), (5, 1000), (33, 1024), (7, 1032),
          (2, 2048), (130, 2056), (16, 4096), (3, 5120), (4, 8192), (3, 8200), (2, 16384),
          (1, 20000), (2, 32768), (1000, 128)]
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _built():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()


def _inputs(rng, tokens, width):
    x = (rng.standard_normal((tokens, width)) * np.exp(rng.standard_normal(width))).astype(np.float16)
    r = (rng.standard_normal((tokens, width)) * 3).astype(np.float16)
    w = (1 + 0.3 * rng.standard_normal(width)).astype(np.float16)
    return x, r, w


def _norm(h, w, eps=EPS):
    h, w = h.astype(np.float64), w.astype(np.float64)
    return h / np.sqrt((h * h).mean(1, keepdims=True) + eps) * w


def _z_error(width):
    return (6 + np.sqrt(width) / 2) * 2.0 ** -23


def _check_codes(Q, z, width):
    """Codes and scales are those of a z that is off by what fp32 allows: each is that of
    z, or of z made a little larger or smaller."""
    d = 4 * _z_error(width)
    codes, scales = [t.cpu().numpy() for t in Q.to_codes()]
    codes = mx_util.unpack(codes, Q.K, Q.format)
    kinds = [mx_util.quantize(z * f, Q.format, 1.0) for f in (1.0, 1.0 + d, 1.0 - d)]
    fits = [scales == k[1] for k in kinds]
    assert np.logical_or.reduce(fits).all()
    # codes are compared where the scale is that of z itself
    same = np.repeat(fits[0], mx_util.BLOCK[Q.format], axis=1)[:, :Q.K]
    assert same.mean() > 0.9
    near = [mx_util.quantize(z * f, Q.format, 1.0) for f in (1.0 + d, 1.0 - d)]
    ok = codes == kinds[0][0]
    for c, s, _ in near:
        ok |= (codes == c) & np.repeat(s == kinds[0][1], mx_util.BLOCK[Q.format],
                                       axis=1)[:, :Q.K]
    assert (ok | ~same).all()
    assert (codes == kinds[0][0])[same].mean() > 0.999


@pytest.mark.parametrize("tokens,width", SHAPES)
@pytest.mark.parametrize("residual", [False, True])
def test_norm(tokens, width, residual):
    import torch

    import tma_pipelined_tensor_fp16_gb300 as tg
    x, r, w = _inputs(np.random.default_rng(tokens + width), tokens, width)
    h = x.astype(np.float64) + (r if residual else 0)
    z = _norm(h, w)
    X, R, W = device(x), device(r) if residual else None, device(w)
    for format in FORMATS:
        Z, H, Q = tg.rms_norm(X, W, residual=R, eps=EPS, format=format)
        torch.cuda.synchronize()
        if residual:
            assert np.array_equal(H.cpu().numpy(), h.astype(np.float16))
        else:
            assert H is X
        tol = _z_error(width) * np.abs(z) + 2.0 ** -11 * np.abs(z) + 2.0 ** -25
        assert_within(Z.cpu().numpy(), z, tol, "Z")
        if format is None:
            assert Q is None
        else:
            _check_codes(Q, z, width)
            alone = tg.rms_norm(X, W, residual=R, eps=EPS, half=False, format=format)
            assert alone[0] is None and torch.equal(alone[2].codes, Q.codes) \
                if tokens % 128 == 0 else all(
                    torch.equal(a, b) for a, b in zip(alone[2].to_codes(), Q.to_codes()))


@pytest.mark.parametrize("width", [
    64, 200, 384, 504, 640, 760, 1000, 1184, 1512, 1968, 2552, 2960, 4088, 4960, 6136, 8000,
    10000, 12240, 16384, 20000])
def test_many_tokens(width):
    """Enough rows for the shapes that long batches take: the rows repeat 37 different ones,
    whose results are compared with 64 bits and must be the same wherever they stand."""
    import torch

    import tma_pipelined_tensor_fp16_gb300 as tg
    tokens, distinct = 152 * 2048 * 8 // width + 131, 37
    x, r, w = _inputs(np.random.default_rng(width), distinct, width)
    h = x.astype(np.float64) + r
    z = _norm(h, w)
    index = torch.arange(tokens, device="cuda") % distinct
    X, R, W = device(x)[index], device(r)[index], device(w)
    for format in FORMATS:
        Z, H, Q = tg.rms_norm(X, W, residual=R, eps=EPS, format=format)
        assert torch.equal(Z, Z[:distinct][index]) and torch.equal(H, H[:distinct][index])
        assert np.array_equal(H[:distinct].cpu().numpy(), h.astype(np.float16))
        tol = _z_error(width) * np.abs(z) + 2.0 ** -11 * np.abs(z) + 2.0 ** -25
        assert_within(Z[:distinct].cpu().numpy(), z, tol, "Z")
        few = tg.rms_norm(X[:distinct], W, residual=R[:distinct], eps=EPS, format=format)
        assert torch.equal(few[0], Z[:distinct])
        if format is not None:
            parts = Q.to_codes()
            assert all(torch.equal(t, t[:distinct][index]) for t in parts)
            assert all(torch.equal(t[:distinct], f) for t, f in zip(parts, few[2].to_codes()))
            _check_codes(tg.MXTensor.from_codes(*(t[:distinct].contiguous() for t in parts),
                                                width, format), z, width)


@pytest.mark.parametrize("width", [72, 384, 640, 1024, 1528, 2048, 3000, 5120, 9472, 16384])
def test_a_rows_gradient_does_not_depend_on_the_others(width):
    import torch

    import tma_pipelined_tensor_fp16_gb300 as tg
    h, dz, w = (device(a) for a in _inputs(np.random.default_rng(width), 3000, width))
    dX, _ = tg.rms_norm_grad(dz, h, w, dH=h)
    for few in (1, 5, 300):
        assert torch.equal(tg.rms_norm_grad(dz[:few], h[:few], w, dH=h[:few])[0], dX[:few])


def test_zero_rows_tiny_rows_and_infinities():
    import torch

    import tma_pipelined_tensor_fp16_gb300 as tg
    x = np.ones((5, 256), np.float16)
    x[0] = 0
    x[1] = 2.0 ** -24
    x[2, 7] = np.inf
    x[3] = 65504
    w = np.ones(256, np.float16)
    Z, _, Q = tg.rms_norm(device(x), device(w), eps=EPS, format="mxfp8")
    Z, V = Z.cpu().numpy(), Q.values().cpu().numpy()
    assert (Z[0] == 0).all() and (V[0] == 0).all()
    assert_within(Z[[1, 3, 4]], _norm(x, w)[[1, 3, 4]], 2e-3, "Z")
    assert np.isnan(Z[2, 7]) and (np.delete(Z[2], 7) == 0).all()
    assert np.isnan(V[2, :32]).all() and (V[2, 32:] == 0).all()
    Z, _, _ = tg.rms_norm(device(x), device(w), eps=0.0)
    assert torch.isnan(Z[0]).all() and torch.isfinite(Z[1]).all()


def test_in_place_streams_and_capture():
    import torch

    import tma_pipelined_tensor_fp16_gb300 as tg
    x, r, w = _inputs(np.random.default_rng(5), 40, 1024)
    X, R, W = device(x), device(r), device(w)
    Z, H, Q = tg.rms_norm(X, W, residual=R, format="nvfp4")
    R2, X2 = R.clone(), X.clone()
    Z2, H2, _ = tg.rms_norm(X2, W, residual=R2, total=R2, out=X2)
    assert H2 is R2 and Z2 is X2 and torch.equal(R2, H) and torch.equal(X2, Z)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    Z3, H3, Q3 = tg.rms_norm(X, W, residual=R, format="nvfp4", stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(Z3, Z) and torch.equal(H3, H) and torch.equal(Q3.values(), Q.values())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        Z4, H4, Q4 = tg.rms_norm(X, W, residual=R, format="nvfp4")
        dX, dw = tg.rms_norm_grad(Z4, H4, W, dH=H4)
    X.mul_(0.5)
    graph.replay()
    Z5, H5, Q5 = tg.rms_norm(X, W, residual=R, format="nvfp4")
    d5, w5 = tg.rms_norm_grad(Z5, H5, W, dH=H5)
    assert torch.equal(Z4, Z5) and torch.equal(H4, H5) and torch.equal(Q4.values(), Q5.values())
    assert torch.equal(dX, d5) and torch.equal(dw, w5)


def _gradient(dz, h, w, dh, eps=EPS):
    dz, h, w = (t.astype(np.float64) for t in (dz, h, w))
    rstd = 1 / np.sqrt((h * h).mean(1, keepdims=True) + eps)
    n, u = h * rstd, dz * w
    dx = rstd * (u - n * (u * n).mean(1, keepdims=True)) + (0 if dh is None else dh)
    return dx, (dz * n).sum(0)


def test_the_formula_against_differences():
    """On the CPU's numbers: the gradient's formula is the derivative of the norm's."""
    rng = np.random.default_rng(1)
    h, w, dz = rng.standard_normal((3, 16)), rng.standard_normal(16), rng.standard_normal((3, 16))
    dx, dw = _gradient(dz, h, w, None)
    step = 1e-6
    for i in (0, 1, 2):
        for j in (0, 7, 15):
            e = np.zeros_like(h)
            e[i, j] = step
            d = ((_norm(h + e, w) - _norm(h - e, w)) * dz).sum() / (2 * step)
            assert abs(d - dx[i, j]) < 1e-7
    for j in (0, 15):
        e = np.zeros_like(w)
        e[j] = step
        assert abs(((_norm(h, w + e) - _norm(h, w - e)) * dz).sum() / (2 * step) - dw[j]) < 1e-7


@pytest.mark.parametrize("tokens,width", SHAPES + [(700, 1024), (2000, 4096), (1, 4096),
                                                   (5000, 264), (3000, 512), (900, 8200),
                                                   (700, 12296), (650, 16384), (400, 32768)])
@pytest.mark.parametrize("residual", [False, True])
def test_gradient(tokens, width, residual):
    """dX: n (u h) is a sum of `width` terms, S = sum |u h|, entering dX through |h| rstd^3 /
    width, and rstd's own error scales every term; dweight: a sum over the tokens whose
    terms are off by rstd's error."""
    import torch

    import tma_pipelined_tensor_fp16_gb300 as tg
    rng = np.random.default_rng(tokens * 3 + width)
    _, h, w = _inputs(rng, tokens, width)
    dz = rng.standard_normal((tokens, width)).astype(np.float16)
    dh = rng.standard_normal((tokens, width)).astype(np.float16) if residual else None
    want, want_w = _gradient(dz, h, w, dh)
    H, W, dZ = device(h), device(w), device(dz)
    dH = device(dh) if residual else None
    dX, dw = tg.rms_norm_grad(dZ, H, W, dH=dH, eps=EPS)
    h64, u = h.astype(np.float64), dz.astype(np.float64) * w
    rstd = 1 / np.sqrt((h64 * h64).mean(1, keepdims=True) + EPS)
    terms = np.abs(u) * rstd + np.abs(h64) * rstd ** 3 * np.abs(u * h64).mean(1, keepdims=True)
    tol = 4 * _z_error(width) * terms + 2.0 ** -11 * np.abs(want) + 2.0 ** -25
    if residual:
        tol += 2.0 ** -23 * np.abs(want)
    assert_within(dX.cpu().numpy(), want, tol, "dX")
    size = (np.abs(dz) * np.abs(h64 * rstd)).sum(0)
    assert_within(dw.cpu().numpy(), want_w,
                  tolerance(want_w, size, tokens, "f32") + _z_error(width) * size, "dweight")
    # again, and in place
    again = tg.rms_norm_grad(dZ, H, W, dH=dH, eps=EPS)
    assert torch.equal(again[0], dX) and torch.equal(again[1], dw)
    to = dZ.clone()
    assert torch.equal(tg.rms_norm_grad(to, H, W, dH=dH, eps=EPS, out=to)[0], dX)


def test_gradient_of_no_tokens():
    import torch

    import tma_pipelined_tensor_fp16_gb300 as tg
    e = torch.empty(0, 64, dtype=torch.float16, device="cuda")
    w = torch.ones(64, dtype=torch.float16, device="cuda")
    dX, dw = tg.rms_norm_grad(e, e, w)
    assert dX.shape == (0, 64) and (dw == 0).all()
    Z, H, Q = tg.rms_norm(e, w, residual=e, format="mxfp4")
    assert Z.shape == H.shape == (0, 64) and Q.rows == 0


def test_offsets_past_32_bits():
    import torch

    import tma_pipelined_tensor_fp16_gb300 as tg
    tokens, width = 540000, 4096
    assert tokens * width > 2 ** 31
    x, r, w = _inputs(np.random.default_rng(11), 3, width)
    X = torch.zeros((tokens, width), dtype=torch.float16, device="cuda")
    X[-3:] = device(x)
    W = device(w)
    Z, _, Q = tg.rms_norm(X, W, eps=1.0, format="mxfp4")
    small = tg.rms_norm(device(x), W, eps=1.0, format="mxfp4")
    assert torch.equal(Z[-3:], small[0]) and int(torch.count_nonzero(Z[:-3])) == 0
    V = Q.values(Z)
    assert torch.equal(V[-3:], small[2].values()) and int(torch.count_nonzero(V[:-3])) == 0
    dX, dw = tg.rms_norm_grad(X, X, W, eps=1.0, out=Z)
    dx, dws = tg.rms_norm_grad(device(x), device(x), W, eps=1.0)
    assert torch.equal(dX[-3:], dx) and int(torch.count_nonzero(dX[:-3])) == 0
    assert torch.allclose(dw, dws, rtol=1e-6, atol=1e-6)
