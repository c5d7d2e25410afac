"""Which stream the memory of the expert operators' tensors belongs to, on stand-ins
for torch and the library (the same on a GPU: test_gpu_expert_streams.py)."""
import pytest

import fake_torch
from fake_torch import Stream, Tensor


@pytest.fixture
def fake(monkeypatch):
    return fake_torch.install(monkeypatch)


def _calls(tg, torch):
    """name -> (a call that takes `stream`, the tensors it is given)."""
    f16, f32, i32, u8 = torch.float16, torch.float32, torch.int32, torch.uint8
    ids, X = Tensor((4, 2), i32), Tensor((4, 64), f16)
    rows, w = Tensor((8, 64), f16), Tensor((4, 2), f32)
    route = tg.ExpertRoute(4, 2, 3).load(Tensor((4,), i32), Tensor((8,), i32), Tensor((4, 2), i32))
    grouped, w4 = tg.GroupedPlan(8, 128, 64, 3), tg.W4Plan(8, 128, 64, group=32, experts=3)
    B, offsets = Tensor((3, 128, 64), f16), Tensor((4,), i32)
    packed, scales = Tensor((3, 128, 32), u8), Tensor((3, 128, 2), f16)
    zeros, each = Tensor((3, 128, 2), u8), Tensor((8,), i32)

    def sort(stream):
        r = tg.ExpertRoute(4, 2, 3).sort(ids, stream=stream)
        return [r.offsets, r.order, r.position]
    return {
        "sort": (sort, [ids]),
        "gather": (lambda s: [route.gather(X, stream=s)], [X, route.offsets, route.position]),
        "combine": (lambda s: [route.combine(rows, weights=w, stream=s)],
                    [rows, w, route.offsets, route.position]),
        "combine_slots": (lambda s: [route.combine_slots(rows, weights=w, stream=s)], [rows, w]),
        "combine_grad": (lambda s: list(route.combine_grad(X, rows, w, stream=s)),
                         [X, rows, w, route.offsets, route.position]),
        "grouped": (lambda s: [grouped(rows, B, offsets, stream=s)], [rows, B, offsets]),
        "w4": (lambda s: [w4(rows, packed, scales, zeros=zeros, ids=each, stream=s)],
               [rows, packed, scales, zeros, each]),
    }


NAMES = ["sort", "gather", "combine", "combine_slots", "combine_grad", "grouped", "w4"]


@pytest.mark.parametrize("name", NAMES)
def test_new_tensors_belong_to_the_stream_that_writes_them(fake, name):
    import tma_pipelined_tensor_fp16_gb300 as tg
    torch, library = fake
    call, inputs = _calls(tg, torch)[name]
    for t in call(Stream(5)):
        assert t.home == 5
    assert library.calls[-1][1][-1] == 5  # the launch
    assert all(t.used_on == {5} for t in inputs)
    assert all(t.home == 1 for t in call(None))
    assert library.calls[-1][1][-1] == 1


def test_tables_are_kept_for_another_stream(fake):
    """The caller never sees a route's tables, so the route keeps them for a stream
    that becomes current after the sort."""
    import tma_pipelined_tensor_fp16_gb300 as tg
    torch, _ = fake
    route = tg.ExpertRoute(4, 2, 3).sort(Tensor((4, 2), torch.int32))
    X = Tensor((4, 64), torch.float16)
    route.gather(X)
    assert not route.offsets.used_on and not X.used_on
    with torch.stream(Stream(9)):
        route.gather(X)
    assert route.offsets.used_on == {9} and route.position.used_on == {9}
    assert not X.used_on  # as everywhere in torch, the caller's
