"""Plans beside others, on stand-ins for torch and the library: the device that each is made
on.  A plan beside none is refused."""
import contextlib

import pytest

import fake_torch


@pytest.fixture(scope="module")
def b():
    from tma_pipelined_tensor_fp16_gb300 import binding, build
    build.build()
    return binding


def test_no_plan(b):
    assert not b.lib().gemm_mx_create_plan_beside(None, 8, 8, 64, 1, 0, 0)
    assert b.gemm_last_status() == b.GEMM_ERR_INVALID_ARG


def test_the_device_of_a_plan(monkeypatch):
    """That of the tensors it is for, whatever the current one is: 0 here."""
    from tma_pipelined_tensor_fp16_gb300 import MXPlan, microscale
    torch, library = fake_torch.install(monkeypatch)
    current, made = [0], []

    @contextlib.contextmanager
    def device(d):
        current.append(d)
        yield
        current.pop()

    class Recorded:
        def __getattr__(self, name):
            if "create" in name:
                made.append((name, current[-1]))
            return getattr(library, name)
    torch.device = device
    monkeypatch.setattr(microscale, "lib", Recorded)
    first = MXPlan(8, 8, 64, device=1)
    MXPlan(16, 8, 64, beside=first)
    MXPlan(8, 8, 64)
    MXPlan(16, 8, 64, beside=MXPlan(8, 8, 64))
    assert [m for m in made if "create" in m[0]] == [
        ("gemm_mx_create_plan_ex", 1), ("gemm_mx_create_plan_beside", 1),
        ("gemm_mx_create_plan_ex", 0), ("gemm_mx_create_plan_ex", 0),
        ("gemm_mx_create_plan_beside", 0)]
