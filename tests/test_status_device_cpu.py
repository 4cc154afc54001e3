"""device_status and the wait checks act on the device that they are given, whichever is the current one.  On the CPU:
torch's notion of the current device and the library are stood in for."""
import contextlib

import pytest
import torch

import kimi_delta_attention_13_gb300 as kda


@pytest.fixture
def world(monkeypatch):
    """[(call, the current device, stream)] of the calls that reach the library; device 0 is current."""
    current, calls = [0], []

    @contextlib.contextmanager
    def device(d):
        before = current[0]
        index = torch.device(d).index
        current[0] = before if index is None else index
        try:
            yield
        finally:
            current[0] = before

    class Lib:
        def __getattr__(self, name):
            def call(*args):
                calls.append((name, current[0], args[-1]))
                return 0
            return call

    monkeypatch.setattr(torch.cuda, "current_device", lambda: current[0])
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 100 + index, raising=False)
    monkeypatch.setattr(kda._lib, "load", Lib)
    return calls


@pytest.mark.parametrize("name", ["device_status", "diag_device_timeout", "diag_linear_timeout", "diag_delta_timeout"])
def test_the_device_that_is_given(world, name):
    call = getattr(kda, name)
    call(device="cuda:1")
    call()
    call(device="cuda")
    call(device=torch.device("cuda", 0))
    assert world == [(f"kda_{name}", 1, 101)] + 3 * [(f"kda_{name}", 0, 100)]
