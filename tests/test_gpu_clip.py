"""The global gradient norm and clipping against numpy in 64 bits.

The norm is the square root of sums that are fp32 over at most 32 squares and fp64 beyond.  Of
the 32, four (eight of fp16, whose squares are exact) are added in turn and those sums in a tree:
seven roundings (nine) of partial sums, so at most 7 * 2^-24 (9, only if each partial sum were the
whole one already; 8 is kept to), and half of it for the norm, plus the norm's own rounding to fp32.
The factor adds one rounding and
each value one of its product and one to its type.
"""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

NORM = 5 * 2.0 ** -24
VALUE = NORM + 2 * 2.0 ** -24
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _built():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()


def _tensor(rng, n, half, scale):
    import torch
    x = (rng.standard_normal(n) * scale).astype(np.float16 if half else np.float32)
    return torch.from_numpy(x).cuda()


def _norm(grads):
    return float(np.sqrt(sum((g.double().cpu().numpy().ravel() ** 2).sum() for g in grads)))


def _check(grads, max_norm, out=None):
    import torch

    import tma_pipelined_tensor_fp16_gb300 as tg
    before = [g.double().cpu().numpy() for g in grads]
    norm = _norm(grads)
    clip = tg.GradClip(grads, out=out)
    alone, got = float(clip.norm()), float(clip(max_norm))
    with np.errstate(over="ignore"):
        held = float(np.float32(norm))  # an infinity where fp32 holds no such number
    for n in (alone, got):
        assert n == held or abs(n - norm) <= NORM * norm
    factor = min(1.0, max_norm / (norm + EPS)) if norm else 1.0
    for b, o in zip(before, grads if out is None else out):
        o16 = o.dtype == torch.float16
        o = o.double().cpu().numpy()
        tol = np.abs(b * factor) * (VALUE + (2.0 ** -11 if o16 else 0))
        tol = tol + (2.0 ** -25 if o16 else 2.0 ** -150)
        assert (np.abs(o - b * factor) <= tol).all()
        if factor == 1.0:
            assert np.array_equal(o, b)
    return norm


@pytest.mark.parametrize("place", ["out", "in place"])
@pytest.mark.parametrize("sizes", [[1], [7], [16384], [16385], [0, 5, 0], [0, 0], [3, 1, 100, 20000, 4096],
                                   list(range(1, 400)), [3000001], [1 << 20] * 5])
def test_sizes_and_types(sizes, place):
    import torch
    rng = np.random.default_rng(len(sizes))
    for mix in (lambda i: False, lambda i: True, lambda i: i % 3 == 0):
        grads = [_tensor(rng, n, mix(i), 0.1) for i, n in enumerate(sizes)]
        out = None if place == "in place" else [torch.empty_like(g) for g in grads]
        norm = _norm(grads)
        _check(grads, 0.3 * norm, out)
        _check(grads, 10.0 * norm, out)  # nothing to clip


def test_views_that_start_anywhere():
    import torch
    rng = np.random.default_rng(0)
    flat, half = _tensor(rng, 100000, False, 1.0), _tensor(rng, 100000, True, 1.0)
    grads = [flat[1:20000], flat[20003:20007], half[1:50], half[57:40000], half[40001:40002]]
    rest = [flat[:1], flat[20000:20003], flat[20007:], half[:1], half[50:57]]
    kept = [t.clone() for t in rest]
    _check(grads, 3.0, [torch.empty(g.numel() + 1, dtype=g.dtype, device="cuda")[1:]
                        for g in grads])
    _check(grads, 3.0)
    assert all(torch.equal(a, b) for a, b in zip(rest, kept))


@pytest.mark.parametrize("scale", [1e-30, 1e-22, 1e-18, 1e15, 1e25, 3e37])
def test_magnitudes_whose_squares_leave_fp32(scale):
    rng = np.random.default_rng(1)
    grads = [_tensor(rng, n, False, scale) for n in (5, 1000, 4099)]
    assert np.isfinite(_norm(grads))
    _check(grads, 0.5 * scale)
    _check([_tensor(rng, 999, False, scale), _tensor(rng, 64, False, 1.0)], 0.25)


def test_infinities_nan_and_zeros():
    import torch

    import tma_pipelined_tensor_fp16_gb300 as tg
    x = torch.ones(100, device="cuda")
    x[3] = float("inf")
    y = torch.ones(50, dtype=torch.float16, device="cuda")
    assert float(tg.clip_grad_norm([x, y], 1.0)) == float("inf")
    assert torch.isnan(x[3]) and (y == 0).all() and int(torch.isnan(x).sum()) == 1
    x[3] = float("nan")
    assert np.isnan(float(tg.clip_grad_norm([x, y], 1.0)))
    assert torch.isnan(x).all() and torch.isnan(y).all()
    z = torch.zeros(1000, device="cuda")
    assert float(tg.clip_grad_norm([z], 0.0, eps=0.0)) == 0.0 and (z == 0).all()
    o = torch.ones(1000, device="cuda")
    tg.clip_grad_norm([o], 0.0)
    assert (o == 0).all()


def test_shapes_streams_and_capture():
    import torch

    import tma_pipelined_tensor_fp16_gb300 as tg
    rng = np.random.default_rng(2)
    grads = [_tensor(rng, 6000, False, 1.0).view(10, 20, 30), _tensor(rng, 512, True, 1.0)]
    out = [torch.empty_like(g) for g in grads]
    clip = tg.GradClip(grads, out=out)
    norm = clip(1.0)
    want = [o.clone() for o in out]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = clip(1.0, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(norm, other) and all(torch.equal(a, b) for a, b in zip(want, out))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = clip(1.0)
    for g in grads:
        g.mul_(2.0)
    graph.replay()
    assert abs(float(held) - 2 * float(norm)) < 1e-3 * float(norm)
    for a, b in zip(want, out):  # clipped to the same length
        assert float((a.double() - b.double()).abs().max()) < 2e-3


def test_refusals():
    import torch

    import tma_pipelined_tensor_fp16_gb300 as tg
    a, b = torch.ones(100, device="cuda"), torch.ones(100, device="cuda")
    for grads, out in (([a, a], None), ([a[:60], a[50:]], None), ([a, b], [b, a]),
                       ([a], [b, b]), ([a[:50]], [a[10:60]]), ([], None)):
        with pytest.raises((ValueError, tg.GemmError)):
            tg.GradClip(grads, out=out)
    with pytest.raises(TypeError):
        tg.GradClip([a.double()])
    with pytest.raises(ValueError):
        tg.GradClip([a.view(10, 10).t()])
    with pytest.raises(ValueError):
        tg.GradClip([a], out=[b[:50]])
    clip = tg.GradClip([a, b])
    for bad in (-1.0, float("nan")):
        with pytest.raises(ValueError):
            clip(bad)
    b.data = torch.ones(100, device="cuda")
    with pytest.raises(ValueError, match="moved"):
        clip(1.0)


def test_offsets_past_32_bits():
    """A tensor of 2^32 + 5 fp16 values, 8.6 GB: only its ends are not zero."""
    import torch

    import tma_pipelined_tensor_fp16_gb300 as tg
    x = torch.zeros(2 ** 32 + 5, dtype=torch.float16, device="cuda")
    x[0], x[-1], x[2 ** 31] = 3.0, 4.0, 12.0
    assert float(tg.clip_grad_norm([x], 1.3)) == 13.0
    for i, v in ((0, 0.3), (-1, 0.4), (2 ** 31, 1.2)):
        assert abs(float(x[i]) - v) < 1e-3
    x[0] = x[-1] = x[2 ** 31] = 0.0
    assert int(torch.count_nonzero(x)) == 0
