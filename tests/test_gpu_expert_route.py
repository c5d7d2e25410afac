"""Tokens sorted by expert and back, against numpy in 64 bits: whole numbers
equal, integer-valued rows bit for bit, random rows within the tolerance of
expert_util, gradients also against differences of the forward operator."""
import numpy as np
import pytest

from expert_util import (assert_same, assert_within, device, integers, normals, routing,
                         sort_reference, tolerance)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()


def _route(ids, experts):
    import tma_pipelined_tensor_fp16_gb300 as tg
    return tg.ExpertRoute(ids.shape[0], ids.shape[1], experts).sort(device(ids))


SHAPES = [  # tokens, topk, experts, drop
    (1, 1, 1, 0.0), (1, 8, 64, 0.0), (3, 2, 5, 0.4), (31, 3, 7, 0.1), (33, 1, 2, 0.0),
    (257, 4, 160, 0.05), (1000, 8, 1024, 0.0), (4097, 2, 3, 0.5), (5000, 6, 257, 0.02),
    (20001, 5, 31, 0.1), (40000, 1, 8, 0.0),
]


@pytest.mark.parametrize("tokens,topk,experts,drop", SHAPES)
def test_sort(tokens, topk, experts, drop):
    rng = np.random.default_rng(tokens * 31 + topk)
    ids = routing(rng, tokens, topk, experts, drop)
    route = _route(ids, experts)
    offsets, order, position = sort_reference(ids, experts)
    assert (route.offsets.cpu().numpy() == offsets).all()
    assert (route.order.cpu().numpy() == order).all()
    assert (route.position.cpu().numpy() == position).all()


@pytest.mark.parametrize("value", [-1, 0, 6, 7])
def test_sort_one_key_only(value):
    """Every slot to one expert, or every slot dropped."""
    ids = np.full((700, 9), value, dtype=np.int32)
    route = _route(ids, 7)
    offsets, order, position = sort_reference(ids, 7)
    assert (route.offsets.cpu().numpy() == offsets).all()
    assert (route.order.cpu().numpy() == order).all()
    assert (route.position.cpu().numpy() == position).all()


def test_sort_repeated_experts_within_a_token():
    rng = np.random.default_rng(5)
    ids = rng.integers(-1, 4, (333, 6)).astype(np.int32)
    route = _route(ids, 4)
    assert (route.order.cpu().numpy() == sort_reference(ids, 4)[1]).all()


def test_no_tokens():
    import torch

    import tma_pipelined_tensor_fp16_gb300 as tg
    route = tg.ExpertRoute(0, 4, 6).sort(torch.empty((0, 4), dtype=torch.int32, device="cuda"))
    assert (route.offsets.cpu().numpy() == 0).all()
    X = torch.empty((0, 64), dtype=torch.float16, device="cuda")
    assert tuple(route.gather(X).shape) == (0, 64)
    assert tuple(route.combine(X).shape) == (0, 64)


WIDTHS = [(1, 4, 9, 0.0, 8), (3, 6, 160, 0.0, 5120), (37, 2, 5, 0.3, 72), (130, 8, 16, 0.05, 1000),
          (65, 20, 40, 0.1, 264), (9, 1, 4, 0.5, 2048), (300, 3, 8, 0.0, 4104)]


@pytest.mark.parametrize("tokens,topk,experts,drop,width", WIDTHS)
def test_gather(tokens, topk, experts, drop, width):
    import torch
    rng = np.random.default_rng(width)
    ids = routing(rng, tokens, topk, experts, drop)
    offsets, order, _ = sort_reference(ids, experts)
    X = normals(rng, (tokens, width))
    X[0, 0], X[-1, -1] = np.inf, np.nan
    out = torch.full((tokens * topk, width), float("nan"), dtype=torch.float16, device="cuda")
    got = _route(ids, experts).gather(device(X), out).cpu().numpy()
    want = X[order // topk].copy()
    want[offsets[-1]:] = 0
    assert np.array_equal(got.view(np.uint16), want.view(np.uint16))


def _combine_reference(Ys, w, ids, experts):
    _, _, position = sort_reference(ids, experts)
    kept = (ids >= 0) & (ids < experts)
    w = np.where(kept, w, 0.0)
    rows = np.where(kept[:, :, None], Ys[position].astype(np.float64), 0.0)
    return (w[:, :, None] * rows).sum(1), np.abs(w[:, :, None] * rows).sum(1)


@pytest.mark.parametrize("out", ["f16", "f32"])
@pytest.mark.parametrize("weighted", [True, False])
@pytest.mark.parametrize("tokens,topk,experts,drop,width", WIDTHS)
def test_combine(tokens, topk, experts, drop, width, weighted, out):
    import torch
    rng = np.random.default_rng(width + topk)
    ids = routing(rng, tokens, topk, experts, drop)
    ids[tokens // 2] = -1  # a token without any slot
    offsets = sort_reference(ids, experts)[0]
    Ys = normals(rng, (tokens * topk, width))
    Ys[offsets[-1]:] = np.nan  # rows of dropped slots are not read
    w = rng.random((tokens, topk)).astype(np.float32) if weighted else \
        np.ones((tokens, topk), np.float32)
    ref, mag = _combine_reference(np.nan_to_num(Ys), w, ids, experts)
    w[(ids < 0) | (ids >= experts)] = np.nan  # nor are their weights
    dt = torch.float16 if out == "f16" else torch.float32
    Y = torch.full((tokens, width), float("nan"), dtype=dt, device="cuda")
    got = _route(ids, experts).combine(device(Ys), Y, weights=device(w) if weighted else None)
    assert_within(got.cpu().numpy(), ref, tolerance(ref, mag, topk, out), "combine")
    assert (got.cpu().numpy()[tokens // 2] == 0).all()


def test_combine_slots():
    """Rows in slot order, no sort."""
    import tma_pipelined_tensor_fp16_gb300 as tg
    rng = np.random.default_rng(3)
    Ys, w = integers(rng, (5 * 3, 40)), rng.integers(0, 4, (5, 3)).astype(np.float32)
    got = tg.ExpertRoute(5, 3, 8).combine_slots(device(Ys), weights=device(w))
    ref = (Ys.astype(np.float64).reshape(5, 3, 40) * w[:, :, None]).sum(1)
    assert_same(got.cpu().numpy(), ref, "f16")


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("tokens,topk,experts,drop,width", WIDTHS)
def test_combine_grad(tokens, topk, experts, drop, width, in_place):
    import torch
    rng = np.random.default_rng(width + 7 * topk)
    ids = routing(rng, tokens, topk, experts, drop)
    ids[tokens // 2] = -1
    offsets, order, position = sort_reference(ids, experts)
    kept = (ids >= 0) & (ids < experts)
    Ys, dY = normals(rng, (tokens * topk, width)), normals(rng, (tokens, width))
    Ys[offsets[-1]:] = np.inf
    w = rng.standard_normal((tokens, topk)).astype(np.float32)
    w[~kept] = np.nan
    Y = device(Ys)
    out = Y if in_place else torch.full_like(Y, float("nan"))
    dYs, dw = _route(ids, experts).combine_grad(device(dY), Y, device(w), out)
    wk = np.where(kept, w, 0.0).astype(np.float64).reshape(-1)
    want = wk[order][:, None] * dY.astype(np.float64)[order // topk]
    assert_within(dYs.cpu().numpy(), want, 2.0 ** -11 * np.abs(want) + 2.0 ** -25
                  + 2.0 ** -23 * np.abs(want), "dYs")
    rows = np.where(kept[:, :, None], np.nan_to_num(Ys, posinf=0.0)[position].astype(np.float64), 0)
    prod = rows * dY.astype(np.float64)[:, None, :]
    assert_within(dw.cpu().numpy(), prod.sum(2),
                  tolerance(prod.sum(2), np.abs(prod).sum(2), width, "f32"), "dweights")


def test_gradients_are_differences():
    """loss = sum(Y * G): a change of one input entry by one changes the loss by
    that entry's gradient, exactly on whole numbers."""
    rng = np.random.default_rng(11)
    T, k, E, W = 6, 3, 4, 16
    ids = routing(rng, T, k, E, 0.2)
    route = _route(ids, E)
    X, G = integers(rng, (T, W)), integers(rng, (T, W))
    Ys, w = integers(rng, (T * k, W)), rng.integers(-2, 3, (T, k)).astype(np.float32)
    H = integers(rng, (T * k, W))

    def loss(Ys, w):
        return (route.combine(device(Ys), weights=device(w)).cpu().numpy().astype(np.float64)
                * G).sum()

    dYs, dw = (x.cpu().numpy() for x in route.combine_grad(device(G), device(Ys), device(w)))
    for r, c in [(0, 0), (5, 3), (T * k - 1, W - 1), (9, 7)]:
        Y2 = Ys.copy()
        Y2[r, c] += 1
        assert loss(Y2, w) - loss(Ys, w) == dYs[r, c]
    for t in range(T):
        for j in range(k):
            w2 = w.copy()
            w2[t, j] += 1
            assert loss(Ys, w2) - loss(Ys, w) == dw[t, j]
    # gather: loss = sum(Xs * H) over the kept rows
    keep = int(route.offsets[-1])
    Hd = H.copy()
    Hd[keep:] = 0
    dX = route.gather_grad(device(H)).cpu().numpy()

    def gloss(X):
        return (route.gather(device(X)).cpu().numpy().astype(np.float64) * Hd).sum()
    for t, c in [(0, 0), (3, 5), (T - 1, W - 1)]:
        X2 = X.copy()
        X2[t, c] += 1
        assert gloss(X2) - gloss(X) == dX[t, c]


def test_other_stream_and_graph():
    import torch
    rng = np.random.default_rng(2)
    ids = routing(rng, 200, 4, 12, 0.1)
    X = integers(rng, (200, 256))
    dids, dX = device(ids), device(X)
    import tma_pipelined_tensor_fp16_gb300 as tg
    route = tg.ExpertRoute(200, 4, 12)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        Y = route.combine(route.sort(dids).gather(dX))
    s.synchronize()
    want = X.astype(np.float64) * ((ids >= 0) & (ids < 12)).sum(1)[:, None]
    assert_same(Y.cpu().numpy(), want, "f16")
    Xs = torch.empty((800, 256), dtype=torch.float16, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        route.sort(dids)
        route.gather(dX, Xs)
        route.combine(Xs, Y)
    dX.neg_()
    for _ in range(3):
        Y.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert_same(Y.cpu().numpy(), -want, "f16")


def test_refusals():
    import torch

    import tma_pipelined_tensor_fp16_gb300 as tg
    route = tg.ExpertRoute(4, 2, 3)
    X = torch.zeros((4, 64), dtype=torch.float16, device="cuda")
    with pytest.raises(RuntimeError, match="not been sorted"):
        route.gather(X)
    ids = torch.zeros((4, 2), dtype=torch.int32, device="cuda")
    with pytest.raises(TypeError):
        route.sort(ids.long())
    with pytest.raises(ValueError):
        route.sort(ids[:3])
    route.sort(ids)
    with pytest.raises(ValueError):
        route.gather(X.t().contiguous().t())
    with pytest.raises(TypeError):
        route.gather(X.float())
    with pytest.raises(tg.GemmError, match="multiple of 8"):
        route.gather(torch.zeros((4, 60), dtype=torch.float16, device="cuda"))
    odd = torch.zeros(4 * 64 + 1, dtype=torch.float16, device="cuda")[1:].view(4, 64)
    with pytest.raises(tg.GemmError, match="16-byte aligned"):
        route.gather(odd)
    with pytest.raises(ValueError):
        route.combine(X)
    with pytest.raises(tg.GemmError, match="1..1024"):
        tg.ExpertRoute(4, 2, 1025).sort(ids)
