"""The expert layer end to end: forward and gradients against the same layer
differentiated in 64 bits, decoding against the layer with the decoded weights."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()


def _reference(X, ids, w, W1, W2):
    """Y in float64 through dense torch operations (differentiable)."""
    import torch
    Y = torch.zeros(X.shape[0], W2.shape[1], dtype=torch.float64, device=X.device)
    for j in range(ids.shape[1]):
        for e in range(W1.shape[0]):
            hit = (ids[:, j] == e).nonzero()[:, 0]
            if hit.numel():
                rows = torch.relu(X[hit] @ W1[e].t()) @ W2[e].t()
                Y = Y.index_add(0, hit, w[hit, j:j + 1] * rows)
    return Y


def _close(got, want, what):
    """fp16 intermediates: each of up to four roundings (2^-11 of the value) is
    spread over a sum, so the error is a small multiple of 2^-11 of the norm."""
    want = want.double()
    err = (got.double() - want).norm() / want.norm()
    assert err < 4 * 2.0 ** -11, (what, float(err))


def test_forward_and_gradients():
    import torch

    from tma_pipelined_tensor_fp16_gb300 import expert_layer
    layer = expert_layer.random_layer(5, 136, 264, 2)
    X, ids, w = expert_layer.random_batch(333, 2, 5, 136)
    ids[3] = -1       # a token without experts
    ids[10, 1] = 77   # a dropped slot
    Y, saved = layer.forward(X, ids, w)
    dY = torch.randn_like(Y)
    X64, w64, A64, B64 = (t.double().requires_grad_() for t in (X, w, layer.W1, layer.W2))
    ref = _reference(X64, ids, w64, A64, B64)
    _close(Y, ref.detach(), "Y")
    assert (Y[3] == 0).all()
    dX, dw, dW1, dW2 = layer.backward(dY, saved)
    ref.backward(dY.double())
    for got, want, what in ((dX, X64.grad, "dX"), (dw, w64.grad, "dweights"),
                            (dW1, A64.grad, "dW1"), (dW2, B64.grad, "dW2")):
        _close(got, want, what)
    assert (dX[3] == 0).all() and (dw[3] == 0).all() and dw[10, 1] == 0


def test_decode_matches_the_decoded_weights():
    import torch

    from tma_pipelined_tensor_fp16_gb300 import expert_layer
    layer = expert_layer.random_layer(6, 256, 512, 3)
    layer.pack(group=64)
    X, ids, w = expert_layer.random_batch(5, 3, 6, 256)
    got = layer.decode(X, ids, w)
    group, p1, p2 = layer._packed

    def decoded(packed, scales, zeros):
        q = torch.stack([packed & 15, packed >> 4], -1).reshape(scales.shape + (group,)).double()
        return ((q - zeros[..., None].double()) * scales[..., None].double()).flatten(-2)
    _close(got, _reference(X.double(), ids, w.double(), decoded(*p1), decoded(*p2)), "decode")


def test_command(capsys):
    from tma_pipelined_tensor_fp16_gb300 import expert_layer
    expert_layer.main(["--tokens", "256", "--width", "256", "--inner", "512", "--steps", "2"])
    out = capsys.readouterr().out
    assert "training step" in out and "decoding step" in out
    assert np.isfinite(float(out.split(" us, ")[1].split(" ")[0]))
