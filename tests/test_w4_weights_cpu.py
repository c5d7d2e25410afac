"""What the 4-bit products of many rows rely on, checked without a device."""
import numpy as np
import pytest


@pytest.fixture(scope="module")
def b():
    from tma_pipelined_tensor_fp16_gb300 import binding, build
    build.build()
    return binding


def test_weights_are_sums_of_two_halves():
    """scale * (q - zero) = hi + lo exactly: hi the product rounded to fp16, lo what is
    left, for every finite scale and every q - zero, -255..15, unless hi overflows."""
    s = np.arange(1 << 15, dtype=np.uint16).view(np.float16)
    s = s[np.isfinite(s)].astype(np.float64)
    for d in range(-255, 16):
        w = s * d  # exact in 64 bits
        with np.errstate(over="ignore"):
            hi = w.astype(np.float16).astype(np.float64)
        fine = np.isfinite(hi)
        lo = (w - hi)[fine]
        assert (lo.astype(np.float16).astype(np.float64) == lo).all()
        assert (np.abs(w[~fine]) > 65504).all()


def test_weights_choice(b):
    import tma_pipelined_tensor_fp16_gb300 as tg
    assert not b.lib().gemm_w4_create_plan_ex(1, 64, 128, 128, 0, 1, 1, 2)
    assert b.gemm_last_status() == b.GEMM_ERR_INVALID_ARG
    with pytest.raises(ValueError, match="weights must be one of"):
        tg.W4Plan(1, 64, 128, weights="fp16")
