"""The experts' grouped products against numpy in 64 bits: integer-valued
operands bit for bit, random ones within the tolerance of expert_util, the
gradients also against differences of the forward product."""
import numpy as np
import pytest

from expert_util import (assert_same, assert_within, device, integers, normals, offsets_of,
                         tolerance)

pytestmark = pytest.mark.gpu

OPS = ["forward", "grad_input", "grad_weight"]


@pytest.fixture(scope="module", autouse=True)
def _built():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()


def _product(op, P, Q, offsets, shape):
    P, Q = P.astype(np.float64), Q.astype(np.float64)
    out = np.zeros(shape)
    for e in range(len(offsets) - 1):
        s = slice(offsets[e], offsets[e + 1])
        if op == "forward":
            out[s] = P[s] @ Q[e].T
        elif op == "grad_input":
            out[s] = P[s] @ Q[e]
        else:
            out[e] = P[s].T @ Q[s]
    return out


def _run(op, rows, N, K, counts, out, make, poison=None, tile="auto"):
    import torch

    import tma_pipelined_tensor_fp16_gb300 as tg
    E = len(counts)
    offsets = offsets_of(counts)
    plan = tg.GroupedPlan(rows, N, K, E, op=op, out=out, tile=tile)
    sp, sq, so = plan.shapes()
    P, Q = make(sp), make(sq)
    got = torch.full((so[0] + 1,) + so[1:], float("nan"), dtype=plan.dtype, device="cuda")
    P2, Q2 = P.copy(), Q.copy()
    if poison is not None:  # rows that belong to no expert
        P2[offsets[-1]:] = poison
        if op == "grad_weight":
            Q2[offsets[-1]:] = poison
    plan(device(P2), device(Q2), device(offsets), got[:-1])
    torch.cuda.synchronize()
    assert plan.device_status() == 0, tg.gemm_last_error() + "; " + plan.describe()
    assert torch.isnan(got[-1]).all(), "wrote past the end"
    want = _product(op, P, Q, offsets, so)
    mag = _product(op, np.abs(P), np.abs(Q), offsets, so)
    n = {"forward": K, "grad_input": N, "grad_weight": max(1, max(counts))}[op]
    return got[:-1].cpu().numpy(), want, tolerance(want, mag, n, out), plan.describe()


CASES = [  # rows, N, K, counts per expert
    (1, 8, 8, [1]),
    (128, 256, 64, [128]),
    (130, 136, 72, [1, 129]),
    (200, 264, 328, [0, 63, 0, 0, 65, 72, 0]),
    (777, 392, 520, [5, 0, 128, 129, 127, 256, 1, 131]),
    (300, 1032, 200, [17, 100, 0, 33, 64]),          # 86 rows belong to no expert
    (64, 512, 1024, [0, 0, 0]),                      # none does
    (1500, 520, 136, [1500]),
    (600, 2056, 1000, [1] * 40 + [0] * 30 + [50, 61, 90, 200]),
]


TILES = ["128x128", "128x256", "256x256"]


@pytest.mark.parametrize("tile", TILES)
@pytest.mark.parametrize("out", ["f16", "f32"])
@pytest.mark.parametrize("op", OPS)
@pytest.mark.parametrize("rows,N,K,counts", CASES)
def test_integers_exact(op, rows, N, K, counts, out, tile):
    rng = np.random.default_rng(N + K)
    got, want, _, what = _run(op, rows, N, K, counts, out, lambda s: integers(rng, s),
                              poison=np.nan, tile=tile)
    assert_same(got, want, out, what)


@pytest.mark.parametrize("tile", TILES)
@pytest.mark.parametrize("op", OPS)
@pytest.mark.parametrize("rows,N,K,counts", [CASES[4], CASES[5], CASES[8]])
def test_random(op, rows, N, K, counts, tile):
    rng = np.random.default_rng(rows)
    for out in ("f16", "f32"):
        got, want, tol, what = _run(op, rows, N, K, counts, out, lambda s: normals(rng, s, 0.5),
                                    poison=np.inf, tile=tile)
        assert_within(got, want, tol, what)


@pytest.mark.parametrize("tile", TILES)
@pytest.mark.parametrize("op", OPS)
def test_another_expert_s_infinity_stays_out(op, tile):
    """A NaN or infinity in one expert's rows or weights reaches no other."""
    import torch

    import tma_pipelined_tensor_fp16_gb300 as tg
    rng = np.random.default_rng(9)
    counts, N, K = [70, 30, 90], 200, 136
    offsets = offsets_of(counts)
    plan = tg.GroupedPlan(190, N, K, 3, op=op, out="f32", tile=tile)
    sp, sq, so = plan.shapes()
    P, Q = integers(rng, sp), integers(rng, sq)
    want = _product(op, P, Q, offsets, so)
    P[70:100] = np.inf
    if op == "grad_weight":
        Q[70:100] = np.nan
    else:
        Q[1] = np.nan
    got = plan(device(P), device(Q), device(offsets)).cpu().numpy()
    torch.cuda.synchronize()
    if op == "grad_weight":
        assert_same(got[[0, 2]], want[[0, 2]], "f32")
    else:
        keep = np.r_[0:70, 100:190]
        assert_same(got[keep], want[keep], "f32")


@pytest.mark.parametrize("tile", TILES)
@pytest.mark.parametrize("op", OPS)
def test_many_tiles_per_cta(op, tile):
    """Enough tiles that every CTA takes several from the counter."""
    rng = np.random.default_rng(4)
    N, K = (2304, 776) if op != "grad_input" else (776, 2304)
    counts = [300, 0, 1, 511, 640, 128, 700, 257, 129, 90]
    got, want, _, what = _run(op, sum(counts) + 44, N, K, counts, "f16",
                              lambda s: integers(rng, s, -1, 1), poison=np.nan, tile=tile)
    assert_same(got, want, "f16", what)


@pytest.mark.parametrize("tile", TILES)
def test_repeated_runs_of_one_plan(tile):
    """The counter starts over with every run, whatever the split was before."""
    import torch

    import tma_pipelined_tensor_fp16_gb300 as tg
    rng = np.random.default_rng(15)
    A, B = integers(rng, (1100, 64)), integers(rng, (7, 1288, 64))
    plan = tg.GroupedPlan(1100, 1288, 64, 7, tile=tile)
    dA, dB = device(A), device(B)
    for _ in range(6):
        counts = rng.multinomial(rng.integers(0, 1101), np.ones(7) / 7)
        C = torch.full((1100, 1288), float("nan"), dtype=torch.float16, device="cuda")
        plan(dA, dB, device(offsets_of(counts)), C)
        torch.cuda.synchronize()
        assert plan.device_status() == 0
        assert_same(C.cpu().numpy(),
                    _product("forward", A, B, offsets_of(counts), (1100, 1288)), "f16")


def test_many_experts():
    rng = np.random.default_rng(6)
    counts = rng.integers(0, 4, 1024).tolist()
    for op in OPS:
        got, want, _, what = _run(op, sum(counts), 64, 72, counts, "f32",
                                  lambda s: integers(rng, s))
        assert_same(got, want, "f32", what)


@pytest.mark.parametrize("op", OPS)
def test_no_rows(op):
    import torch

    import tma_pipelined_tensor_fp16_gb300 as tg
    plan = tg.GroupedPlan(0, 64, 128, 5, op=op, out="f32")
    sp, sq, so = plan.shapes()
    z = lambda s: torch.zeros(s, dtype=torch.float16, device="cuda")
    out = torch.full(so, float("nan"), dtype=torch.float32, device="cuda")
    plan(z(sp), z(sq), torch.zeros(6, dtype=torch.int32, device="cuda"), out)
    assert (out == 0).all()


def test_offsets_out_of_range_are_clamped():
    """A table that leaves [0, rows] or descends gives wrong rows, no fault."""
    import torch

    import tma_pipelined_tensor_fp16_gb300 as tg
    z = torch.ones((40, 64), dtype=torch.float16, device="cuda")
    w = torch.ones((3, 64, 64), dtype=torch.float16, device="cuda")
    bad = torch.tensor([-5, 30, 10, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    for op in OPS:
        plan = tg.GroupedPlan(40, 64, 64, 3, op=op, out="f32")
        plan(z, z if op == "grad_weight" else w, bad)
        torch.cuda.synchronize()
        assert plan.device_status() == 0


def test_gradients_are_differences():
    """loss = sum(C * G): the gradients are the loss's differences, exactly."""
    import tma_pipelined_tensor_fp16_gb300 as tg
    rng = np.random.default_rng(12)
    counts, N, K = [5, 0, 9, 3], 24, 16
    R, E = sum(counts), len(counts)
    offsets = device(offsets_of(counts))
    A, B, G = integers(rng, (R, K)), integers(rng, (E, N, K)), integers(rng, (R, N))
    fwd = tg.GroupedPlan(R, N, K, E, "forward", "f32")
    dA = tg.GroupedPlan(R, N, K, E, "grad_input", "f32")(device(G), device(B), offsets)
    dB = tg.GroupedPlan(R, N, K, E, "grad_weight", "f32")(device(G), device(A), offsets)
    dA, dB = dA.cpu().numpy(), dB.cpu().numpy()

    def loss(A, B):
        return (fwd(device(A), device(B), offsets).cpu().numpy().astype(np.float64) * G).sum()
    base = loss(A, B)
    for r, k in [(0, 0), (4, 15), (5, 3), (16, 7)]:
        A2 = A.copy()
        A2[r, k] += 1
        assert loss(A2, B) - base == dA[r, k]
    for e, n, k in [(0, 0, 0), (1, 3, 3), (2, 23, 15), (3, 8, 9)]:
        B2 = B.copy()
        B2[e, n, k] += 1
        assert loss(A, B2) - base == dB[e, n, k]


def test_graph_and_stream():
    import torch

    import tma_pipelined_tensor_fp16_gb300 as tg
    rng = np.random.default_rng(13)
    A, B = integers(rng, (300, 128)), integers(rng, (3, 256, 128))
    plan = tg.GroupedPlan(300, 256, 128, 3)
    offs = device(offsets_of([100, 150, 50]))
    dA, dB = device(A), device(B)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    C = torch.empty((300, 256), dtype=torch.float16, device="cuda")
    plan(dA, dB, offs, C, stream=s)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        plan(dA, dB, offs, C)
    for counts in ([10, 0, 290], [299, 1, 0]):  # a replay reads the offsets anew
        offs.copy_(device(offsets_of(counts)))
        C.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert_same(C.cpu().numpy(), _product("forward", A, B, offsets_of(counts), (300, 256)),
                    "f16")


def test_refusals():
    import torch

    import tma_pipelined_tensor_fp16_gb300 as tg
    with pytest.raises(tg.GemmError, match="multiples of 8"):
        tg.GroupedPlan(16, 60, 64, 2)
    with pytest.raises(tg.GemmError, match="1..1024"):
        tg.GroupedPlan(16, 64, 64, 1025)
    with pytest.raises(ValueError):
        tg.GroupedPlan(16, 64, 64, 2, op="backward")
    with pytest.raises(ValueError):
        tg.GroupedPlan(16, 64, 64, 2, out="bf16")
    with pytest.raises(ValueError):
        tg.GroupedPlan(16, 64, 64, 2, tile="64x64")
    with pytest.raises(tg.GemmError, match="so many experts"):
        tg.GroupedPlan(16, 64, 64, 1024, tile="256x256")
    plan = tg.GroupedPlan(16, 64, 64, 2)
    z = lambda *s: torch.zeros(s, dtype=torch.float16, device="cuda")
    offs = torch.zeros(3, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        plan(z(15, 64), z(2, 64, 64), offs)
    with pytest.raises(TypeError):
        plan(z(16, 64), z(2, 64, 64), offs.long())
    with pytest.raises(ValueError):
        plan(z(16, 64), z(2, 64, 64).transpose(1, 2), offs)
    odd = torch.zeros(16 * 64 + 1, dtype=torch.float16, device="cuda")[1:].view(16, 64)
    with pytest.raises(tg.GemmError, match="16-byte aligned"):
        plan(odd, z(2, 64, 64), offs)
