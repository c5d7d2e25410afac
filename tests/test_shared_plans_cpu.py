"""The plans that a shared expert keeps while its batches change their length."""
import gc
import weakref

import pytest
import torch


class Plan:
    """A product in plain torch; `all` holds the plans that live."""
    all = weakref.WeakSet()

    def __init__(self, M, N, K, format="mxfp8", out="f16", beside=None, device=None):
        assert beside is not None or device is not None
        self.sizes, self.format, self.beside = (M, N, K), format, beside
        Plan.all.add(self)

    def device_status(self):
        return 4

    def __call__(self, A, B, out=None):
        assert (A.shape[0], B.shape[0], A.shape[1]) == self.sizes
        return A @ B.t() if out is None else out.copy_(A @ B.t())


@pytest.fixture
def shared(monkeypatch):
    from tma_pipelined_tensor_fp16_gb300 import expert_layer

    class Q(torch.Tensor):
        rows = property(lambda self: self.shape[0])
    monkeypatch.setattr(expert_layer, "MXPlan", Plan)
    monkeypatch.setattr(expert_layer, "mx_quantize", lambda x, format, transpose=False, out=None:
                        (x.t() if transpose else x).clone().as_subclass(Q))
    gc.collect()
    Plan.all.clear()
    made = expert_layer.SharedExpert(torch.randn(16, 8), torch.randn(8, 16))
    made.Q = Q
    return made


def test_few_are_kept_and_one_has_the_memory(shared):
    for tokens in range(1, 150):
        x = torch.randn(tokens, 8)
        Y, A = shared.forward(x.as_subclass(shared.Q))
        shared.backward(Y, A, x)
        assert len(Plan.all) <= 65
    assert [p.beside for p in Plan.all].count(None) == 1
    assert shared.device_status() == 4 and len(shared.plans()) == 1


def test_nothing_keeps_it_alive(shared):
    """Its plans go with it, not when the collector next runs."""
    from tma_pipelined_tensor_fp16_gb300 import expert_layer
    other = expert_layer.SharedExpert(shared.S1, shared.S2)
    other.forward(torch.randn(3, 8).as_subclass(shared.Q))
    gc.disable()
    try:
        before = len(Plan.all)
        del other
        assert len(Plan.all) == before - 3
    finally:
        gc.enable()
