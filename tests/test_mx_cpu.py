"""The block-scaled and layer operators without a device: argument checks of the C entry
points, storage sizes, the storage order of row-major codes, and the formats' arithmetic in
mx_util against their definition."""
import ctypes

import numpy as np
import pytest

import mx_util

LIM = (1 << 31) - 65536
FORMATS = {"mxfp8": 0, "mxfp4": 1, "nvfp4": 2}


@pytest.fixture(scope="module")
def b():
    from tma_pipelined_tensor_fp16_gb300 import binding, build
    build.build()
    return binding


def _sizes(b, rows, K, format):
    c, s = ctypes.c_int64(), ctypes.c_int64()
    status = b.lib().gemm_mx_sizes(rows, K, format, ctypes.byref(c), ctypes.byref(s))
    return status, c.value, s.value


@pytest.mark.parametrize("name", FORMATS)
def test_sizes(b, name):
    from tma_pipelined_tensor_fp16_gb300 import microscale
    for rows, K in ((0, 1), (1, 1), (128, 64), (129, 65), (1000, 4097), (5, 96), (5, 97)):
        packed = np.zeros((rows, K if name == "mxfp8" else -(-K // 2)), np.uint8)
        scales = np.zeros((rows, -(-K // mx_util.BLOCK[name])), np.uint8)
        c, s = mx_util.storage(packed, scales, K, name)
        assert _sizes(b, rows, K, FORMATS[name]) == (0, c.size, s.size)
        assert microscale._shapes(rows, K, name) == (c.shape, s.shape)


def test_size_refusals(b):
    assert _sizes(b, 8, 64, 3)[0] == b.GEMM_ERR_INVALID_ARG
    assert _sizes(b, -1, 64, 0)[0] == b.GEMM_ERR_INVALID_ARG
    assert _sizes(b, 8, 0, 0)[0] == b.GEMM_ERR_INVALID_ARG
    assert _sizes(b, LIM + 1, 64, 0)[0] == b.GEMM_ERR_INVALID_ARG
    assert _sizes(b, LIM, LIM, 0)[0] == b.GEMM_ERR_UNSUPPORTED


def test_quantize_refusals(b):
    q = b.lib().gemm_mx_quantize
    X, C, S, T = 4096, 8192, 12288, 16384  # never read: each call is refused
    for args, status in (
            ((8, 64, 9, 0, X, C, S, None, None), b.GEMM_ERR_INVALID_ARG),
            ((8, 60, 0, 0, X, C, S, None, None), b.GEMM_ERR_UNSUPPORTED),
            ((12, 64, 0, 1, X, C, S, None, None), b.GEMM_ERR_UNSUPPORTED),
            ((8, 64, 0, 0, X, C, S, T, None), b.GEMM_ERR_INVALID_ARG),
            ((8, 64, 2, 0, X, C, S, None, None), b.GEMM_ERR_INVALID_ARG),
            ((8, 64, 0, 0, None, C, S, None, None), b.GEMM_ERR_INVALID_ARG),
            ((8, 64, 0, 0, X + 2, C, S, None, None), b.GEMM_ERR_UNSUPPORTED),
            ((8, 64, 2, 0, X, C, S, T + 2, None), b.GEMM_ERR_UNSUPPORTED)):
        assert q(*args, None) == status, args
    v = b.lib().gemm_mx_values
    for args, status in (
            ((8, 64, 0, C, S, None, 7, X), b.GEMM_ERR_INVALID_ARG),
            ((8, 64, 0, C, S, T, 1, X), b.GEMM_ERR_INVALID_ARG),
            ((8, 64, 0, C, None, None, 1, X), b.GEMM_ERR_INVALID_ARG),
            ((8, 64, 0, C, S, None, 1, X + 8), b.GEMM_ERR_UNSUPPORTED)):
        assert v(*args, None) == status, args


def test_plan_refusals(b):
    make = b.lib().gemm_mx_create_plan_ex
    for args, status in (
            ((8, 8, 64, 5, 1, 0, 0), b.GEMM_ERR_INVALID_ARG),
            ((0, 8, 64, 0, 1, 0, 0), b.GEMM_ERR_INVALID_ARG),
            ((8, 8, 0, 0, 1, 0, 0), b.GEMM_ERR_INVALID_ARG),
            ((8, LIM + 8, 64, 0, 1, 0, 0), b.GEMM_ERR_INVALID_ARG),
            ((8, 8, 64, 0, 2, 0, 0), b.GEMM_ERR_INVALID_ARG),
            ((8, 8, 64, 0, 1, 9, 0), b.GEMM_ERR_INVALID_ARG),
            ((8, 8, 64, 0, 1, 0, 3), b.GEMM_ERR_INVALID_ARG),
            ((8, 12, 64, 0, 1, 0, 0), b.GEMM_ERR_UNSUPPORTED),
            ((8, 6, 64, 0, 0, 0, 0), b.GEMM_ERR_UNSUPPORTED),
            ((8, 1 << 24, 1 << 24, 0, 1, 0, 0), b.GEMM_ERR_UNSUPPORTED)):
        assert not make(*args) and b.gemm_last_status() == status, args
    run = b.lib().gemm_mx_run
    assert run(None, 16, 16, None, 16, 16, None, 16, None) == b.GEMM_ERR_INVALID_ARG
    assert b.lib().gemm_mx_set_wait(None, 0, 0) == b.GEMM_ERR_INVALID_ARG
    assert b.lib().gemm_mx_get_device_status(None) == b.GEMM_ERR_INVALID_ARG
    b.lib().gemm_mx_destroy(None)


def test_norm_refusals(b):
    f = b.lib().gemm_rms_norm
    X, W, Z = 4096, 8192, 12288
    ok = dict(tokens=4, width=64, X=X, R=None, w=W, eps=1e-6, H=None, Z=Z, f=0, c=None, s=None)
    for change, status in (
            (dict(tokens=-1), b.GEMM_ERR_INVALID_ARG), (dict(width=60), b.GEMM_ERR_UNSUPPORTED),
            (dict(width=0), b.GEMM_ERR_UNSUPPORTED), (dict(width=32776), b.GEMM_ERR_UNSUPPORTED),
            (dict(eps=-1.0), b.GEMM_ERR_INVALID_ARG),
            (dict(eps=float("nan")), b.GEMM_ERR_INVALID_ARG),
            (dict(X=None), b.GEMM_ERR_INVALID_ARG), (dict(w=None), b.GEMM_ERR_INVALID_ARG),
            (dict(Z=None), b.GEMM_ERR_INVALID_ARG), (dict(H=Z), b.GEMM_ERR_INVALID_ARG),
            (dict(c=X), b.GEMM_ERR_INVALID_ARG), (dict(c=X, s=X, f=4), b.GEMM_ERR_INVALID_ARG),
            (dict(X=X + 2), b.GEMM_ERR_UNSUPPORTED)):
        assert f(*{**ok, **change}.values(), None) == status, change
    g = b.lib().gemm_rms_norm_grad
    assert g(4, 64, X, X, W, None, 1e-6, Z, None, X, None) == b.GEMM_ERR_INVALID_ARG
    assert g(4, 64, X, X, W, None, 1e-6, Z, W, None, None) == b.GEMM_ERR_INVALID_ARG
    assert g(4, 64, X, X + 8, W, None, 1e-6, Z, W, X, None) == b.GEMM_ERR_UNSUPPORTED
    assert b.lib().gemm_rms_norm_grad_workspace(4, 60) == -1
    for tokens, width in ((0, 8), (1, 64), (100000, 128), (100000, 4096), (3, 32768)):
        assert b.lib().gemm_rms_norm_grad_workspace(tokens, width) % (4 * width) == 0


def _clip(b, grads, outs, sizes, types):
    n = len(grads)
    p = ctypes.c_void_p * n
    made = b.lib().gemm_clip_create_plan(n, p(*grads), p(*outs), (ctypes.c_int64 * n)(*sizes),
                                         (ctypes.c_int * n)(*types))
    assert not made
    return b.gemm_last_status()


def test_clip_refusals(b):
    """Outputs that share memory are refused before a device is looked for."""
    import torch
    M = 1 << 20
    apart = b.GEMM_ERR_NO_DEVICE
    if not torch.cuda.is_available():
        assert _clip(b, [M, 2 * M], [M, 2 * M], [100, 100], [0, 1]) == apart
        assert _clip(b, [M, M + 400], [M, M + 400], [100, 100], [0, 0]) == apart
        assert _clip(b, [M, M], [3 * M, 4 * M], [100, 100], [0, 0]) == apart
        assert _clip(b, [M, 0], [M, 0], [100, 0], [0, 0]) == apart
    bad = b.GEMM_ERR_INVALID_ARG
    assert _clip(b, [M, M], [M, M], [100, 100], [0, 0]) == bad
    assert _clip(b, [M, M + 396], [M, M + 396], [100, 100], [0, 0]) == bad
    assert _clip(b, [M, 2 * M], [2 * M, M], [100, 100], [0, 0]) == bad
    assert _clip(b, [M], [M + 4], [100], [0]) == bad
    assert _clip(b, [M, 3 * M], [2 * M, 2 * M + 196], [100, 100], [1, 0]) == bad
    assert _clip(b, [M, 4 * M], [3 * M, 3 * M - 1000], [5000, 300], [0, 0]) == bad
    assert _clip(b, [M], [M], [-1], [0]) == bad
    assert _clip(b, [M], [M], [5], [2]) == bad
    assert _clip(b, [None], [None], [5], [0]) == bad
    assert _clip(b, [M + 2], [M + 2], [5], [0]) == b.GEMM_ERR_UNSUPPORTED
    run = b.lib().gemm_clip_run
    assert run(None, 1.0, 1e-6, M, M, None) == bad
    assert run(None, -1.0, 1e-6, M, M, None) == bad
    assert b.lib().gemm_clip_norm(None, M, M, None) == bad
    b.lib().gemm_clip_destroy(None)


def test_rounding_of_the_reference():
    """Every midpoint of the formats goes to the even code, and a hair beside it does not."""
    for format, levels in (("mxfp4", mx_util.E2M1), ("mxfp8", mx_util.e4m3_values()[:127])):
        mid = (levels[1:] + levels[:-1]) / 2
        even = np.where(np.arange(len(mid)) % 2 == 0, np.arange(len(mid)), np.arange(len(mid)) + 1)
        assert (mx_util.nearest(mid, levels) == even).all()
        assert (mx_util.nearest(mid * (1 + 1e-12), levels) == np.arange(1, len(levels))).all()
        assert (mx_util.nearest(mid * (1 - 1e-12), levels) == np.arange(len(mid))).all()
        assert (mx_util.nearest(levels, levels) == np.arange(len(levels))).all()
        assert mx_util.nearest(np.array([1e9]), levels)[0] == len(levels) - 1


def test_scales_of_the_reference():
    for largest in (448.0, 6.0, 2688.0):
        for e in (-40, -1, 0, 3, 15):
            top = largest * 2.0 ** e
            got = mx_util.power_of_two(np.array([top, top * (1 + 1e-9), top / 2, top * 0.51]), largest)
            assert got.tolist() == [e, e + 1, e - 1, e]
    codes, scales, t = mx_util.quantize(np.array([[448.0] + [0.0] * 31, [1.0] * 32]), "mxfp8")
    assert scales.tolist() == [[127], [119]] and codes[0, 0] == 0x7e and codes[1, 0] == 0x78


@pytest.mark.parametrize("name,rows,K", [("mxfp8", 130, 100), ("mxfp4", 260, 72), ("mxfp4", 3, 200),
                                         ("nvfp4", 40, 264), ("nvfp4", 3, 35)])
def test_row_major_codes_and_storage(monkeypatch, name, rows, K):
    """The storage order from its description, on CPU tensors (the device check aside)."""
    import torch

    from tma_pipelined_tensor_fp16_gb300 import microscale
    monkeypatch.setattr(microscale, "_tensor", lambda what, t, *rest: t)
    packed, scales, _, _ = mx_util.random_operand(np.random.default_rng(K), rows, K, name, True)
    Q = microscale.MXTensor.from_codes(torch.from_numpy(packed), torch.from_numpy(scales), K, name)
    c, s = mx_util.storage(packed, scales, K, name)
    assert (Q.codes.numpy() == c).all() and (Q.scales.numpy() == s).all()
    back = Q.to_codes()
    assert (back[0].numpy() == packed).all() and (back[1].numpy() == scales).all()


def test_cpu_tensors_are_refused():
    import torch

    import tma_pipelined_tensor_fp16_gb300 as tg
    x = torch.zeros(8, 64, dtype=torch.float16)
    with pytest.raises(ValueError):
        tg.mx_quantize(x)
    with pytest.raises(ValueError):
        tg.rms_norm(x, x[0])
    with pytest.raises(ValueError):
        tg.rms_norm_grad(x, x, x[0])
    with pytest.raises(ValueError):
        tg.GradClip([x])
    with pytest.raises(ValueError):
        tg.mx_quantize(x, "fp8")
    with pytest.raises(ValueError):
        tg.MXPlan(8, 8, 64, format="mxfp6")
    with pytest.raises(ValueError):
        tg.MXPlan(8, 8, 64, kernel="fast")
