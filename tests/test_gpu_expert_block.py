"""A block of the model end to end: the norm, the experts' layer, the shared expert in a
block-scaled format, their gradients and clipping, against 64 bits on the values that the
quantised operands stand for."""
import pytest

from test_gpu_expert_layer import _close, _reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()


def _block(format, tokens=333):
    from tma_pipelined_tensor_fp16_gb300 import expert_layer
    block = expert_layer.random_block(5, 136, 264, 2, 200, format)
    X, ids, w = expert_layer.random_batch(tokens, 2, 5, 136)
    return block, X, X.flip(0).contiguous(), ids, w


def _rounded(x, format, transpose=False):
    """The 64-bit values of fp16 x rounded to the format (along its columns)."""
    import torch

    import tma_pipelined_tensor_fp16_gb300 as tg
    Q = tg.mx_quantize(x, format, transpose=transpose)
    V = Q.values(torch.empty((Q.rows, Q.K), dtype=torch.float32, device="cuda")).double()
    return V.t() if transpose else V


@pytest.mark.parametrize("format", ["mxfp8", "mxfp4", "nvfp4"])
def test_forward_and_gradients(format):
    import torch
    block, X, R, ids, w = _block(format)
    layer, shared = block.layer, block.shared
    Y, H, saved = block.forward(X, R, ids, w)
    _, Z, A, _ = saved
    h = X.double() + R.double()
    rstd = (h.square().mean(1, keepdim=True) + block.eps).rsqrt()
    _close(Z, h * rstd * block.norm_weight.double(), "Z")
    assert torch.equal(H, h.half())
    # the shared expert, from the quantised norm on (its codes are of the unrounded norm)
    import tma_pipelined_tensor_fp16_gb300 as tg
    Q = tg.rms_norm(X, block.norm_weight, residual=R, eps=block.eps, half=False, format=format)[2]
    q = Q.values(torch.empty(Z.shape, dtype=torch.float32, device="cuda")).double()
    _close(A, torch.relu(q @ _rounded(shared.S1, format).t()), "A")
    S = _rounded(A, format) @ _rounded(shared.S2, format).t()
    routed = _reference(Z.double(), ids, w.double(), layer.W1.double(), layer.W2.double())
    _close(Y, routed + S, "Y")

    dY, dH = torch.randn_like(Y), torch.randn_like(H)
    dX, dw = block.backward(dY, dH, saved)
    leaves = [t.double().requires_grad_() for t in (Z, w, layer.W1, layer.W2)]
    _reference(leaves[0], ids, *leaves[1:]).backward(dY.double())
    _close(dw, leaves[1].grad, "dweights")
    _close(block.grads[0], leaves[2].grad, "dW1")
    _close(block.grads[1], leaves[3].grad, "dW2")
    dA = (_rounded(dY, format) @ _rounded(shared.S2, format, True)).half()
    dHs = dA.masked_fill(A <= 0, 0.0)
    _close(block.grads[3], _rounded(dY, format, True).t() @ _rounded(A, format, True), "dS2")
    _close(block.grads[2], _rounded(dHs, format, True).t() @ _rounded(Z, format, True), "dS1")
    dS = _rounded(dHs, format) @ _rounded(shared.S1, format, True)
    # from here on fp16 roundings of the parts of dZ are amplified by the norm's subtraction
    dZ = leaves[0].grad + dS
    n, u = H.double() * rstd, dZ * block.norm_weight.double()
    _close(dX, dH.double() + rstd * (u - n * (u * n).mean(1, keepdim=True)), "dX")
    _close(block.grads[4], (dZ * n).sum(0), "dnorm")

    want = [g.clone() for g in block.grads]
    norm = float(sum(g.double().square().sum() for g in want).sqrt())
    assert abs(float(block.clip(0.25 * norm)) - norm) < 1e-6 * norm
    for g, b in zip(block.grads, want):
        assert float((g - 0.25 * b).norm()) <= 1e-5 * float(b.norm())
    assert block.device_status() == 0


def test_update_lays_the_weights_out_again():
    import torch
    block, X, R, ids, w = _block("mxfp8", tokens=64)
    first, _, saved = block.forward(X, R, ids, w)
    block.backward(first, None, saved)
    block.clip(1.0)
    block.update(0.5)
    second = block.forward(X, R, ids, w)[0]
    again = block.forward(X, R, ids, w)[0]
    assert not torch.equal(first, second) and torch.equal(second, again)


def test_decode():
    import torch
    from tma_pipelined_tensor_fp16_gb300 import expert_layer
    block = expert_layer.random_block(6, 256, 512, 3, 384, "nvfp4")
    block.layer.pack(group=64)
    X, ids, w = expert_layer.random_batch(5, 3, 6, 256)
    Y, H = block.decode(X, X, ids, w)
    Z = __import__("tma_pipelined_tensor_fp16_gb300").rms_norm(X, block.norm_weight, residual=X)[0]
    full, _, (_, _, _, _) = block.forward(X, X, ids, w)
    shared = full.double() - block.layer.forward(Z, ids, w)[0].double()
    _close(Y, block.layer.decode(Z, ids, w).double() + shared, "decode")
    assert torch.equal(H, (X.float() * 2).half())
    none = block.decode(X[:0], X[:0], ids[:0], w[:0])
    assert none[0].shape == none[1].shape == (0, 256)


def test_no_tokens():
    import torch
    block, X, R, ids, w = _block("nvfp4")
    Y, H, saved = block.forward(X[:0], R[:0], ids[:0], w[:0])
    for g in block.grads:
        g.fill_(7.0)
    dX, dw = block.backward(Y, None, saved)
    assert Y.shape == H.shape == dX.shape == (0, 136) and dw.shape == (0, 2)
    assert all((g == 0).all() for g in block.grads) and float(block.clip(1.0)) == 0.0


def test_a_step_in_a_graph():
    """Forward, backward and clipping captured and replayed, against the calls."""
    import torch
    block, X, R, ids, w = _block("mxfp4", tokens=128)

    def step():
        Y, H, saved = block.forward(X, R, ids, w)
        out = block.backward(Y, H, saved)
        return (Y, H) + out + (block.clip(1.0),)
    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    X.mul_(0.5)
    graph.replay()
    got = [t.clone() for t in held] + [g.clone() for g in block.grads]
    want = list(step()) + block.grads
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_command_runs_the_block(capsys):
    from tma_pipelined_tensor_fp16_gb300 import expert_layer
    expert_layer.main(["--tokens", "256", "--width", "256", "--inner", "512", "--steps", "2",
                       "--shared", "384", "--format", "nvfp4"])
    out = capsys.readouterr().out
    assert "block's training step" in out and "block's decoding step" in out
