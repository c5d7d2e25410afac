"""Argument checks of the expert-layer entry points that need no device, and the
arithmetic the kernels rely on, checked on the CPU.  Every call here is refused
before a launch: none passes the checks with an address that is not real."""
import numpy as np
import pytest

from expert_util import routing, sort_reference


@pytest.fixture(scope="module")
def b():
    from tma_pipelined_tensor_fp16_gb300 import binding, build
    build.build()
    return binding


@pytest.mark.parametrize("args,status", [
    ((-1, 2, 4), 1), ((4, 0, 4), 1), ((4, 257, 4), 1), ((4, 2, 0), 1), ((4, 2, 1025), 1),
    ((1 << 30, 2, 4), 2), ((4, 2, 4), 1),  # the last: NULL pointers
])
def test_sort_arguments(b, args, status):
    assert b.lib().gemm_expert_sort(*args, None, None, None, None, None) == status
    assert b.last_error()


def test_row_arguments(b):
    L = b.lib()
    assert L.gemm_expert_gather(4, 2, 4, 60, None, None, None, None, None) == b.GEMM_ERR_UNSUPPORTED
    assert L.gemm_expert_gather(4, 2, 4, 64, None, None, None, None, None) == b.GEMM_ERR_INVALID_ARG
    assert L.gemm_expert_gather(4, 2, 4, 64, 8, 16, 16, 16, None) == b.GEMM_ERR_UNSUPPORTED
    assert L.gemm_expert_combine(4, 2, 4, 64, 16, None, None, None, 7, 16, None) == \
        b.GEMM_ERR_INVALID_ARG
    assert L.gemm_expert_combine(4, 2, 4, 64, 16, None, 16, None, 1, 16, None) == \
        b.GEMM_ERR_INVALID_ARG
    assert L.gemm_expert_combine_grad(4, 2, 4, 64, 16, 16, 16, 16, None, 16, 16, None) == \
        b.GEMM_ERR_INVALID_ARG
    # nothing to do, nothing checked on the device
    assert L.gemm_expert_gather(0, 2, 4, 64, None, None, None, None, None) == b.GEMM_OK


@pytest.mark.parametrize("args,status", [
    ((16, 64, 64, 2, 0, 2), 1), ((16, 64, 64, 2, 3, 0), 1), ((-1, 64, 64, 2, 0, 0), 1),
    ((16, 60, 64, 2, 0, 0), 2), ((16, 64, 60, 2, 0, 0), 2), ((16, 64, 64, 0, 0, 0), 1),
    ((16, 1 << 30, 64, 2, 0, 0), 2),
])
def test_grouped_arguments(b, args, status):
    assert not b.lib().gemm_grouped_create_plan(*args)
    assert b.gemm_last_status() == status
    assert b.lib().gemm_grouped_run(None, None, None, None, None, None) == b.GEMM_ERR_INVALID_ARG


@pytest.mark.parametrize("args,status", [
    ((1, 64, 256, 48, 0, 1, 1), 1), ((1, 64, 192, 128, 0, 1, 1), 2), ((1, 60, 128, 128, 0, 1, 1), 2),
    ((0, 64, 128, 128, 0, 1, 1), 1), ((1, 64, 128, 128, 0, 2, 1), 1),
    ((1025, 64, 128, 128, 4, 1, 1), 2),
])
def test_w4_arguments(b, args, status):
    assert not b.lib().gemm_w4_create_plan(*args)
    assert b.gemm_last_status() == status
    assert b.lib().gemm_w4_run(None, None, None, None, None, None, None, None) == \
        b.GEMM_ERR_INVALID_ARG


def test_wrappers_refuse_host_tensors():
    import torch

    import tma_pipelined_tensor_fp16_gb300 as tg
    with pytest.raises(ValueError, match="contiguous CUDA tensor"):
        tg.ExpertRoute(2, 2, 4).sort(torch.zeros((2, 2), dtype=torch.int32))
    with pytest.raises(ValueError):
        tg.ExpertRoute(2, 0, 4)
    with pytest.raises(RuntimeError, match="not been sorted"):
        tg.ExpertRoute(2, 2, 4).gather(torch.zeros((2, 8), dtype=torch.float16))


def test_codes_become_exact_halves():
    """1024 + q and 1024 + 16 q, less the zero point, are exact in fp16 for every
    code and every zero point 0..255."""
    q = np.arange(16)[:, None]
    z = np.arange(256)[None, :]
    low = (1024 + q).astype(np.float16) + (-1024.0 - z).astype(np.float16)
    assert (low == q - z).all()
    high = (1024 + 16 * q).astype(np.float16) * np.float16(0.0625)  # exact: 64 + q
    assert (high == 64 + q).all()
    assert (high + (-64.0 - z).astype(np.float16) == q - z).all()


def test_warp_order_of_the_sort():
    """Rows by (key, earlier CTAs and warps, earlier lanes) are the stable sort's,
    for the run lengths the launch uses."""
    rng = np.random.default_rng(0)
    for tokens, topk, experts in [(5, 3, 4), (700, 2, 9), (3000, 4, 33)]:
        ids = routing(rng, tokens, topk, experts, 0.1).reshape(-1)
        slots = ids.size
        ctas = 1
        while ctas < 8 and slots > 4096 * ctas:
            ctas *= 2
        warps = 32
        while warps > 8 and slots <= warps * 32 * ctas:
            warps //= 2
        run = (-(-slots // (ctas * warps)) + 31) // 32 * 32
        key = np.where((ids < 0) | (ids >= experts), experts, ids)
        counts = np.zeros((ctas * warps, experts + 1), dtype=int)
        for w in range(ctas * warps):
            np.add.at(counts[w], key[w * run:(w + 1) * run], 1)
        start = np.concatenate([[0], np.cumsum(counts.sum(0))[:-1]])
        at = start + np.cumsum(counts, 0) - counts
        position = np.empty(slots, dtype=int)
        for w in range(ctas * warps):
            for s in range(w * run, min((w + 1) * run, slots)):
                position[s] = at[w, key[s]]
                at[w, key[s]] += 1
        assert (position == sort_reference(ids, experts)[2]).all()
