"""Quantisation to the block-scaled formats and back, bit for bit against numpy: every
rounding is decided by arithmetic that 64 bits hold exactly."""
import numpy as np
import pytest

import mx_util
from expert_util import device

pytestmark = pytest.mark.gpu

FORMATS = ["mxfp8", "mxfp4", "nvfp4"]


@pytest.fixture(scope="module", autouse=True)
def _built():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()


def _check(Q, x, t=None):
    """Q against the 64-bit quantisation of x (rows x K)."""
    import torch
    codes, scales, t = mx_util.quantize(x.astype(np.float64), Q.format, t)
    torch.cuda.synchronize()
    got_c, got_s = [v.cpu().numpy() for v in Q.to_codes()]
    assert (got_s == scales).all()
    if Q.format == "nvfp4":
        assert float(Q.tensor_scale) == t
    bad = np.repeat(scales == (127 if Q.format == "nvfp4" else 255),
                    mx_util.BLOCK[Q.format], axis=1)[:, :Q.K]
    got_c = mx_util.unpack(got_c, Q.K, Q.format)
    assert ((got_c == codes) | bad).all()
    # behind the row's end: zeros (of either sign is not enough: bytes of zero)
    width = got_c.shape[1] if Q.format == "mxfp8" else -(-Q.K // 2)
    tail = Q.codes.permute(0, 2, 1, 3).reshape(Q.codes.shape[0] * 128, -1)[:Q.rows, width:]
    assert int(tail.max()) == 0 if tail.numel() else True
    # values
    want = mx_util.values(codes, scales, Q.format, t)
    full = Q.values(torch.empty(Q.rows, Q.K, device="cuda")).cpu().numpy()
    half = Q.values().cpu().numpy()
    assert np.array_equal(full.astype(np.float64), want, equal_nan=True)
    with np.errstate(over="ignore"):
        assert np.array_equal(half, want.astype(np.float32).astype(np.float16), equal_nan=True)


def _inputs(rng, rows, K):
    """Values of all sizes, blocks of zeros, exact ties, the largest and smallest halves."""
    x = rng.standard_normal((rows, K)) * 2.0 ** rng.integers(-12, 12, (rows, 1))
    x = x * np.exp(rng.standard_normal((1, K)))
    x = np.where(rng.random((rows, K)) < 0.1, rng.integers(-24, 25, (rows, K)) / 4.0, x)
    x = x.astype(np.float16)
    if K >= 64:
        x[::3, :32] = 0.0
        x[1::3, 32:64] = np.float16(2.0 ** -24)
    x[::5, -1] = np.float16(65504.0)
    return np.where(np.isfinite(x), x, np.float16(-60000.0))


SHAPES = [(1, 8), (1, 128), (3, 40), (7, 264), (33, 96), (64, 512), (127, 136), (128, 64),
          (129, 1000), (200, 4096), (5, 16384), (1030, 72)]


@pytest.mark.parametrize("format", FORMATS)
@pytest.mark.parametrize("rows,K", SHAPES)
def test_along_rows(format, rows, K):
    import tma_pipelined_tensor_fp16_gb300 as tg
    x = _inputs(np.random.default_rng(rows * 7 + K), rows, K)
    _check(tg.mx_quantize(device(x), format), x)


@pytest.mark.parametrize("format", FORMATS)
@pytest.mark.parametrize("rows,K", [(8, 1), (8, 33), (40, 127), (64, 128), (72, 129), (136, 500),
                                    (1000, 77), (4096, 31), (264, 4097)])
def test_along_columns(format, rows, K):
    import tma_pipelined_tensor_fp16_gb300 as tg
    x = _inputs(np.random.default_rng(rows * 5 + K), rows, K)
    _check(tg.mx_quantize(device(x.T.copy()), format, transpose=True), x)


@pytest.mark.parametrize("format", FORMATS)
@pytest.mark.parametrize("transpose", [False, True])
def test_infinities_and_nan_stay_in_their_block(format, transpose):
    import tma_pipelined_tensor_fp16_gb300 as tg
    x = _inputs(np.random.default_rng(9), 40, 200)
    x[3, 5], x[3, 70], x[8, 199], x[9, 0], x[9, 1] = np.inf, np.nan, -np.inf, np.nan, np.inf
    X = device(x.T.copy() if transpose else x)
    Q = tg.mx_quantize(X, format, transpose=transpose)
    _check(Q, x)
    v = Q.values().cpu().numpy()
    block = mx_util.BLOCK[format]
    assert np.isnan(v[3, :block]).all() and np.isnan(v[9, :block]).all()
    assert np.isfinite(v[3, block:2 * block]).all() and np.isfinite(v[4]).all()


def test_every_half_rounds_as_defined():
    """All finite halves as rows of blocks that they lead, and mixed at random."""
    import tma_pipelined_tensor_fp16_gb300 as tg
    h = np.arange(65536, dtype=np.uint16).view(np.float16)
    h = h[np.isfinite(h)]
    h = np.concatenate([h, np.zeros(-h.size % 128, np.float16)])
    rng = np.random.default_rng(4)
    for x in (h.reshape(-1, 128), rng.permutation(h).reshape(-1, 128)):
        for format in FORMATS:
            _check(tg.mx_quantize(device(x), format), x)


@pytest.mark.parametrize("t", [2.0 ** -6, 1.0, 2.0 ** 5])
def test_given_tensor_scale(t):
    import torch

    import tma_pipelined_tensor_fp16_gb300 as tg
    x = (np.random.default_rng(3).standard_normal((50, 320)) * 3).astype(np.float16)
    scale = torch.tensor([t], device="cuda")
    _check(tg.mx_quantize(device(x), "nvfp4", tensor_scale=scale), x, t)
    y = x[:48]
    _check(tg.mx_quantize(device(y.T.copy()), "nvfp4", transpose=True, tensor_scale=scale), y, t)
    assert float(scale) == t


def test_a_given_scale_stays_the_callers():
    """Quantising again into the same tensor finds a scale of its own."""
    import torch

    import tma_pipelined_tensor_fp16_gb300 as tg
    rng = np.random.default_rng(5)
    x = (rng.standard_normal((20, 64)) * 300).astype(np.float16)
    scale = torch.tensor([0.25], device="cuda")
    Q = tg.mx_quantize(device(x), "nvfp4", tensor_scale=scale)
    assert Q.tensor_scale is scale
    _check(tg.mx_quantize(device(x), "nvfp4", out=Q), x)
    assert float(scale) == 0.25 and Q.tensor_scale is not scale
    packed, scales, _, _ = mx_util.random_operand(rng, 20, 64, "nvfp4", True)
    R = tg.MXTensor.from_codes(device(packed), device(scales), 64, "nvfp4", scale)
    _check(tg.mx_quantize(device(x), "nvfp4", out=R), x)
    assert float(scale) == 0.25


def test_zeros_and_no_rows():
    import torch

    import tma_pipelined_tensor_fp16_gb300 as tg
    for format in FORMATS:
        _check(tg.mx_quantize(torch.zeros(10, 64, dtype=torch.float16, device="cuda"), format),
               np.zeros((10, 64)))
        Q = tg.mx_quantize(torch.zeros(0, 64, dtype=torch.float16, device="cuda"), format)
        assert Q.values().shape == (0, 64)
        if format == "nvfp4":
            assert float(Q.tensor_scale) == 1.0


def test_out_is_written_again_and_other_streams():
    import torch

    import tma_pipelined_tensor_fp16_gb300 as tg
    rng = np.random.default_rng(8)
    side = torch.cuda.Stream()
    for format in FORMATS:
        x, y = (_inputs(rng, 70, 264) for _ in range(2))
        Q = tg.mx_quantize(device(x), format)
        assert tg.mx_quantize(device(y), format, out=Q) is Q
        _check(Q, y)
        X = device(x)
        side.wait_stream(torch.cuda.current_stream())
        R = tg.mx_quantize(X, format, stream=side)
        v = R.values(stream=side)
        torch.cuda.current_stream().wait_stream(side)
        _check(R, x)
        assert torch.equal(v, R.values())


def test_captured_and_replayed():
    import torch

    import tma_pipelined_tensor_fp16_gb300 as tg
    rng = np.random.default_rng(2)
    x, y = (_inputs(rng, 130, 264) for _ in range(2))
    X = device(x)
    tg.mx_quantize(X, "nvfp4")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        Q = tg.mx_quantize(X, "nvfp4")
        T = tg.mx_quantize(X, "mxfp8", transpose=True)
    for v in (x, y):
        X.copy_(device(v))
        graph.replay()
        _check(Q, v)
        _check(T, v.T)


def test_storage_order_and_row_major_codes():
    import tma_pipelined_tensor_fp16_gb300 as tg
    rng = np.random.default_rng(6)
    for format, rows, K in (("mxfp8", 130, 100), ("mxfp4", 260, 72), ("nvfp4", 40, 264),
                            ("nvfp4", 3, 35)):
        packed, scales, _, _ = mx_util.random_operand(rng, rows, K, format, True)
        Q = tg.MXTensor.from_codes(device(packed), device(scales), K, format)
        c, s = mx_util.storage(packed, scales, K, format)
        assert (Q.codes.cpu().numpy() == c).all() and (Q.scales.cpu().numpy() == s).all()
        back = Q.to_codes()
        assert (back[0].cpu().numpy() == packed).all() and (back[1].cpu().numpy() == scales).all()


@pytest.mark.parametrize("transpose", [False, True])
def test_offsets_past_32_bits(transpose):
    """2.2e9 values: the last rows and columns are those of the small matrix that they hold."""
    import torch

    import tma_pipelined_tensor_fp16_gb300 as tg
    rows, K = (65600, 33536)
    assert rows * K > 2 ** 31
    X = torch.zeros((rows, K), dtype=torch.float16, device="cuda")
    x = _inputs(np.random.default_rng(1), 64, 128)
    X[-64:, -128:] = device(x)
    want = x.T.copy() if transpose else x
    for format in ("mxfp8", "nvfp4"):
        Q = tg.mx_quantize(X, format, transpose=transpose)
        codes, scales, t = mx_util.quantize(want.astype(np.float64), format)
        ref = mx_util.values(codes, scales, format, t)
        V = Q.values(torch.empty((Q.rows, Q.K), dtype=torch.float32, device="cuda"))
        end = V[-want.shape[0]:, -want.shape[1]:]
        assert np.array_equal(end.double().cpu().numpy(), ref)
        assert int((V[:-want.shape[0]] != 0).sum()) == 0
        assert int((V[:, :-want.shape[1]] != 0).sum()) == 0
        del V, Q


@pytest.mark.parametrize("format", ["mxfp8", "mxfp4", "nvfp4"])
@pytest.mark.parametrize("width", [256, 260, 289])
def test_values_of_every_code_and_scale(format, width):
    """fp16 values are the exact products, rounded once: those that fp32 holds.  The rows' lengths
    let them start anywhere."""
    import torch

    import tma_pipelined_tensor_fp16_gb300 as tg
    rng = np.random.default_rng(width)
    rows, per = 256, 1 if format == "mxfp8" else 2
    block = 16 if format == "nvfp4" else 32
    codes = torch.from_numpy(np.stack([rng.permutation(256) for _ in range(rows)] * 2, 1)
                             .reshape(rows, 512)[:, :-(-width // per)].astype(np.uint8)).cuda()
    scales = torch.arange(rows, device="cuda").to(torch.uint8)[:, None].repeat(1, -(-width // block))
    scales[:, 1::2] = scales[:, 1::2] ^ 1
    for t in [None] if format != "nvfp4" else [2.0 ** -126, 2.0 ** -16, 2.0 ** -15, 2.0 ** -9, 1.0,
                                               2.0 ** 7, 2.0 ** 8, 2.0 ** 100, 0.75]:
        scale = None if t is None else torch.tensor([t], dtype=torch.float32, device="cuda")
        Q = tg.MXTensor.from_codes(codes.contiguous(), scales, width, format, scale)
        full = Q.values(torch.empty(rows, width, device="cuda"))
        half, want = Q.values(), full.half()
        same = (half.view(torch.int16) == want.view(torch.int16)) | (half.isnan() & want.isnan())
        assert bool(same.all()), (t, int((~same).sum()))
        assert bool((full.isnan() == half.isnan()).all())
