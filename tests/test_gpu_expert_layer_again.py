"""The expert layer called again and at its edges."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()


def test_backward_twice():
    import torch

    from tma_pipelined_tensor_fp16_gb300 import expert_layer
    layer = expert_layer.random_layer(4, 64, 128, 2)
    X, ids, w = expert_layer.random_batch(50, 2, 4, 64)
    Y, saved = layer.forward(X, ids, w)
    first = layer.backward(Y, saved)
    for a, b in zip(first, layer.backward(Y, saved)):
        assert torch.equal(a, b)


def test_pack_again_with_another_group():
    from tma_pipelined_tensor_fp16_gb300 import expert_layer
    layer = expert_layer.random_layer(4, 128, 256, 2)
    X, ids, w = expert_layer.random_batch(3, 2, 4, 128)
    want, _ = layer.forward(X, ids, w)
    for group in (128, 32, 64, 128):
        layer.pack(group=group)
        got = layer.decode(X, ids, w)
        assert (got.float() - want.float()).norm() < 0.4 * want.float().norm()


def test_no_tokens():
    import torch

    from tma_pipelined_tensor_fp16_gb300 import expert_layer
    layer = expert_layer.random_layer(4, 64, 128, 2)
    layer.pack(group=64)
    X, ids, w = expert_layer.random_batch(3, 2, 4, 64)
    X, ids, w = X[:0], ids[:0], w[:0]
    Y, saved = layer.forward(X, ids, w)
    dX, dw, dW1, dW2 = layer.backward(Y, saved)
    torch.cuda.synchronize()
    assert Y.shape == dX.shape == layer.decode(X, ids, w).shape == (0, 64)
    assert (dW1 == 0).all() and (dW2 == 0).all()


def test_decode_ignores_what_a_dropped_slot_holds():
    import torch

    from tma_pipelined_tensor_fp16_gb300 import expert_layer
    layer = expert_layer.random_layer(4, 128, 256, 3)
    layer.pack(group=64)
    X, ids, w = expert_layer.random_batch(5, 3, 4, 128)
    ids[0, 1], ids[3] = -1, 4
    clean = layer.decode(X, ids, w)
    w[0, 1] = w[3, 0] = float("nan")
    w[3, 1] = float("inf")
    assert torch.equal(layer.decode(X, ids, w), clean)
    assert torch.isfinite(clean).all() and (clean[3] == 0).all()
