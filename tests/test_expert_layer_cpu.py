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
