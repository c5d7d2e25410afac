"""mx_quantize into an MXTensor of the caller's, on stand-ins for torch and the library: which
tensor scale the result has, and where that lies."""
import pytest

import fake_torch
from fake_torch import Tensor


@pytest.fixture
def fake(monkeypatch):
    from tma_pipelined_tensor_fp16_gb300 import microscale
    torch, library = fake_torch.install(monkeypatch)
    monkeypatch.setattr(microscale, "lib", lambda: library)
    return torch, library


def _tensor(torch, own):
    """An nvfp4 MXTensor of 20 x 64, in the library's memory or the caller's."""
    from tma_pipelined_tensor_fp16_gb300 import microscale as m
    if own:
        return m.MXTensor._new(20, 64, "nvfp4", Tensor.device, None)
    codes, scales = (Tensor(s, torch.uint8) for s in m._shapes(20, 64, "nvfp4"))
    return m.MXTensor(20, 64, "nvfp4", codes, scales, Tensor((1,), torch.float32))


@pytest.mark.parametrize("own", [False, True])
@pytest.mark.parametrize("was_given", [False, True])
@pytest.mark.parametrize("given", [False, True])
def test_a_call_that_fails_leaves_the_scale(fake, monkeypatch, own, was_given, given):
    from tma_pipelined_tensor_fp16_gb300 import GemmError, build
    from tma_pipelined_tensor_fp16_gb300 import microscale as m
    build.build()  # the error has the library's message
    torch, library = fake
    X, f32 = Tensor((20, 64), torch.float16), torch.float32
    Q = _tensor(torch, own)
    m.mx_quantize(X, "nvfp4", out=Q, tensor_scale=Tensor((1,), f32) if was_given else None)
    before = Q._addresses()
    with monkeypatch.context() as patch:
        patch.setattr(library, "gemm_mx_quantize", lambda *args: 1, raising=False)
        with pytest.raises(GemmError):
            m.mx_quantize(X, "nvfp4", out=Q, tensor_scale=Tensor((1,), f32) if given else None)
    assert Q._addresses() == before


@pytest.mark.parametrize("own", [False, True])
def test_a_found_scale_keeps_its_place(fake, own):
    """A captured product reads the scale where it was: quantising again writes it there, also
    after a call with a scale of the caller's."""
    from tma_pipelined_tensor_fp16_gb300 import microscale as m
    torch, library = fake
    X = Tensor((20, 64), torch.float16)
    Q = _tensor(torch, own)
    first = m.mx_quantize(X, "nvfp4", out=Q)._addresses()
    assert m.mx_quantize(X, "nvfp4", out=Q)._addresses() == first
    given = Tensor((1,), torch.float32)
    assert m.mx_quantize(X, "nvfp4", out=Q, tensor_scale=given)._addresses()[2] == given.address
    assert m.mx_quantize(X, "nvfp4", out=Q)._addresses() == first
    name, args = library.calls[-1]
    assert name == "gemm_mx_quantize" and args[7] == first[2]
