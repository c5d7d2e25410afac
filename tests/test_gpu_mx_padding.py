"""What lies behind the K values of a quantised row: codes of zero with scales that are
numbers, whoever wrote the row, for the product's last step multiplies them.  The memory
holds 0xFF before (codes and scales of NaN, or the largest magnitude of e2m1)."""
import numpy as np
import pytest

import mx_util
from expert_util import assert_within, device

pytestmark = pytest.mark.gpu

FORMATS = ["mxfp8", "mxfp4", "nvfp4"]
CODE = {"mxfp8": 0, "mxfp4": 1, "nvfp4": 2}
# each side of a step of the norm's lanes and vectors, and the largest rows: rows of mxfp4
# are filled up to 96 values, past 32768 from 32744 on
WIDTHS = [8, 72, 128, 136, 256, 264, 384, 512, 520, 640, 768, 776, 1024, 1032, 1280, 1536, 2040,
          2056, 2560, 3000, 4096, 4104, 5120, 6144, 8184, 8200, 10240, 12288, 16376, 16392,
          20480, 20488, 24576, 32736, 32744, 32752, 32760, 32768]


@pytest.fixture(scope="module", autouse=True)
def _built():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()


def _poisoned(rows, K, format):
    """Storage of a rows x K matrix, every byte 0xFF, as an MXTensor of its own."""
    import torch

    import tma_pipelined_tensor_fp16_gb300 as tg
    from tma_pipelined_tensor_fp16_gb300 import microscale
    parts = [torch.full(shape, 255, dtype=torch.uint8, device="cuda")
             for shape in microscale._shapes(rows, K, format)]
    return tg.MXTensor(rows, K, format, *parts)


def _check_behind(Q, what):
    blocks, chunks, _, _ = Q.codes.shape
    codes = Q.codes.permute(0, 2, 1, 3).reshape(blocks * 128, chunks * 16)[:Q.rows]
    used = Q.K if Q.format == "mxfp8" else -(-Q.K // 2)
    assert int((codes[:, used:] != 0).sum()) == 0, what
    per_group = 3 if Q.format == "mxfp4" else 4
    scales = Q.scales.permute(0, 3, 2, 1, 4)[..., :per_group].reshape(blocks * 128, -1)[:Q.rows]
    behind = scales[:, -(-Q.K // mx_util.BLOCK[Q.format]):]
    nan = (behind & 127) == 127 if Q.format == "nvfp4" else behind == 255
    assert int(nan.sum()) == 0, what


def _norm_into(Q, X, W):
    import torch

    import tma_pipelined_tensor_fp16_gb300 as tg
    from tma_pipelined_tensor_fp16_gb300 import binding
    status = binding.lib().gemm_rms_norm(
        Q.rows, Q.K, X.data_ptr(), None, W.data_ptr(), 1e-6, None, None, CODE[Q.format],
        Q.codes.data_ptr(), Q.scales.data_ptr(), torch.cuda.current_stream().cuda_stream)
    assert status == 0, tg.gemm_last_error()


@pytest.mark.parametrize("format", FORMATS)
@pytest.mark.parametrize("width", WIDTHS)
def test_norm(width, format):
    import torch
    rng = np.random.default_rng(width)
    many = 152 * 2048 * 8 // width + 3  # rows for the shapes of long batches
    x = device(rng.standard_normal((37, width)).astype(np.float16))
    w = torch.ones(width, dtype=torch.float16, device="cuda")
    for rows in (3, many):
        X = x[torch.arange(rows, device="cuda") % 37].contiguous()
        Q = _poisoned(rows, width, format)
        _norm_into(Q, X, w)
        _check_behind(Q, (rows, width))
        assert bool(Q.values()[:, -8:].isfinite().all())


@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("format", FORMATS)
@pytest.mark.parametrize("rows,K", [(8, 8), (40, 72), (136, 264), (8, 4104), (16, 32744),
                                    (8, 32768)])
def test_quantiser(rows, K, format, transpose):
    import torch

    import tma_pipelined_tensor_fp16_gb300 as tg
    x = device(np.random.default_rng(K).standard_normal((rows, K)).astype(np.float16))
    Q = _poisoned(rows, K, format)
    X = x.t().contiguous() if transpose else x
    assert tg.mx_quantize(X, format, transpose=transpose, out=Q) is Q
    _check_behind(Q, (rows, K))
    assert bool(Q.values(torch.empty(rows, K, device="cuda")).isfinite().all())


@pytest.mark.parametrize("format", FORMATS)
@pytest.mark.parametrize("width", [200, 1032, 32744, 32768])
def test_product_of_the_norms_rows(width, format):
    """Rows as the norm left them, multiplied with each other's and with the quantiser's.

    A row's product with itself has terms of one sign, whose additions may all be truncated
    the same way, so that their errors add up: each of the n additions is off by at most
    2^-23 of a partial sum, and that is at most S = sum |a b|, hence n * 2^-23 * S."""
    import torch

    import tma_pipelined_tensor_fp16_gb300 as tg
    rng = np.random.default_rng(width + 1)
    X = device(rng.standard_normal((72, width)).astype(np.float16))
    W = torch.ones(width, dtype=torch.float16, device="cuda")
    Q = _poisoned(72, width, format)
    _norm_into(Q, X, W)
    P = tg.mx_quantize(X[:24].contiguous(), format)
    q = Q.values(torch.empty(72, width, device="cuda")).double().cpu().numpy()
    p = P.values(torch.empty(24, width, device="cuda")).double().cpu().numpy()
    for A, a in ((Q, q), (P, p)):
        for kernel in ("pair", "single"):
            C = tg.MXPlan(A.rows, 72, width, format=format, out="f32", kernel=kernel)(A, Q)
            ref, size = a @ q.T, np.abs(a) @ np.abs(q).T
            assert_within(C.cpu().numpy(), ref, width * 2.0 ** -23 * size, kernel)
