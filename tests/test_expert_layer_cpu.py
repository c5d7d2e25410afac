"""What ExpertLayer does around the operators, with plain torch in their place."""
import pytest
import torch

import layer_doubles


@pytest.fixture(autouse=True)
def _doubles(monkeypatch):
    layer_doubles.install(monkeypatch)


def test_backward_leaves_what_forward_saved():
    """A second backward from the same forward, as a retained graph needs it."""
    layer, X, ids, w = layer_doubles.layer()
    Y, saved = layer.forward(X, ids, w)
    before = [t.clone() for t in saved if isinstance(t, torch.Tensor)]
    first = layer.backward(Y, saved)
    for t, b in zip((t for t in saved if isinstance(t, torch.Tensor)), before):
        assert torch.equal(t, b)
    for a, b in zip(first, layer.backward(Y, saved)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("value", [float("inf"), float("nan")])
def test_masked_gradient_is_zero_whatever_it_was(value):
    """One token's gradient is not finite: the units that its relu masks out get none
    of it."""
    layer, X, ids, w = layer_doubles.layer()
    Y, saved = layer.forward(X, ids, w)
    clean = layer.backward(Y, saved)
    dY = Y.clone()
    dY[2, 0] = value
    _, _, dW1, _ = layer.backward(dY, saved)
    route, _, H = saved[:3]
    off = {(e, i): False for e in range(layer.experts) for i in range(layer.inner)}
    for j in range(layer.topk):
        e, row = int(ids[2, j]), int(route.position[2, j])
        for i in range(layer.inner):
            off[e, i] |= bool(H[row, i] > 0)
    for (e, i), touched in off.items():
        if not touched:
            assert torch.isfinite(dW1[e, i]).all()
        else:
            assert not torch.isfinite(dW1[e, i]).all()
    assert all(torch.isfinite(t).all() for t in clean)


def test_pack_again_with_another_group():
    layer, X, ids, w = layer_doubles.layer(width=128, inner=128)
    want, _ = layer.forward(X, ids, w)
    for group in (128, 32, 64, 128):
        layer.pack(group=group)
        got = layer.decode(X, ids, w)
        assert (got - want).norm() < 0.4 * want.norm()


def test_no_tokens():
    layer, X, ids, w = layer_doubles.layer()
    layer.pack(group=32)
    X, ids, w = X[:0], ids[:0], w[:0]
    Y, saved = layer.forward(X, ids, w)
    assert Y.shape == (0, 32)
    dX, dw, dW1, dW2 = layer.backward(Y, saved)
    assert dX.shape == (0, 32) and (dW1 == 0).all() and (dW2 == 0).all()
    assert layer.decode(X, ids, w).shape == (0, 32)


def test_decode_ignores_what_a_dropped_slot_holds():
    """As forward does: a routing weight that is not a number counts for nothing there."""
    layer, X, ids, w = layer_doubles.layer()
    layer.pack(group=32)
    ids[0, 1], ids[3] = -1, layer.experts
    clean = layer.decode(X, ids, w)
    w = w.clone()
    w[0, 1] = w[3, 0] = float("nan")
    w[3, 1] = float("inf")
    assert torch.equal(layer.decode(X, ids, w), clean)
    assert (clean[3] == 0).all()
    assert torch.isfinite(layer.forward(X, ids, w)[0]).all()


def test_device_status_is_that_of_every_plan(monkeypatch):
    """A wait that ran out in any of the layer's kernels is reported."""
    layer, X, ids, w = layer_doubles.layer()
    assert layer.device_status() == 0
    layer.pack(group=32)
    Y, saved = layer.forward(X, ids, w)
    layer.backward(Y, saved)
    layer.decode(X, ids, w)
    plans = layer.plans()
    assert len(plans) >= 6
    for i, plan in enumerate(plans):
        monkeypatch.setattr(plan, "device_status", lambda: 4, raising=False)
        assert layer.device_status() == 4
        monkeypatch.setattr(plan, "device_status", lambda: 0, raising=False)


def test_decode_before_pack_says_so():
    layer, X, ids, w = layer_doubles.layer()
    with pytest.raises(RuntimeError, match="call pack"):
        layer.decode(X, ids, w)
