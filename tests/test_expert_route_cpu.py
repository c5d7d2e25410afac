"""Whose tables a route writes, on stand-ins for torch and the library."""
import pytest

import fake_torch
from fake_torch import Tensor


@pytest.fixture
def fake(monkeypatch):
    return fake_torch.install(monkeypatch)


def _written(library):
    """Addresses of the last sort's offsets, order and position."""
    name, args = library.calls[-1]
    assert name == "gemm_expert_sort"
    return set(args[4:7])


def test_sort_leaves_loaded_tables_alone(fake):
    import tma_pipelined_tensor_fp16_gb300 as tg
    torch, library = fake
    mine = [Tensor((4,), torch.int32), Tensor((8,), torch.int32), Tensor((4, 2), torch.int32)]
    ids = Tensor((4, 2), torch.int32)
    route = tg.ExpertRoute(4, 2, 3).load(*mine)
    route.sort(ids)
    assert not _written(library) & {t.address for t in mine}
    first = _written(library)
    route.sort(ids)  # its own, again
    assert _written(library) == first == {t.address for t in (route.offsets, route.order,
                                                              route.position)}
    route.load(*mine).sort(ids)
    assert not _written(library) & {t.address for t in mine}
