"""What rms_norm returns as h when z takes the place of an input, on stand-ins for torch and the
library."""
import pytest

import fake_torch
from fake_torch import Tensor


@pytest.fixture
def torch(monkeypatch):
    from tma_pipelined_tensor_fp16_gb300 import layer, microscale
    fake, library = fake_torch.install(monkeypatch)
    for module in (layer, microscale):
        monkeypatch.setattr(module, "lib", lambda: library)
    return fake


def test_h_is_not_what_z_has_overwritten(torch):
    """Without a residual h is X: once z lies there, there is none that a gradient could take."""
    from tma_pipelined_tensor_fp16_gb300 import rms_norm
    X, R, W = (Tensor(s, torch.float16) for s in ((4, 64), (4, 64), (64,)))
    view = Tensor((4, 64), torch.float16)
    view.address = X.address
    for out in (X, view):
        Z, H, _ = rms_norm(X, W, out=out)
        assert Z is out and H is None
    assert rms_norm(X, W)[1] is X and rms_norm(X, W, out=R)[1] is X
    assert rms_norm(X, W, half=False, format="mxfp8")[1] is X
    for out in (X, R):  # with one, h has memory of its own
        assert rms_norm(X, W, residual=R, out=out)[1].address not in (X.address, R.address)
    assert rms_norm(X, W, residual=R, out=X, total=R)[1] is R


def test_no_tokens(torch):
    from tma_pipelined_tensor_fp16_gb300 import rms_norm
    X, W = Tensor((0, 64), torch.float16), Tensor((64,), torch.float16)
    assert rms_norm(X, W, out=X)[1] is X
