"""Which device and stream the binding calls the library on, where the tensors are not on the current device (stand-ins
for torch's device state and the library; no GPU is touched)."""
import types

import pytest
import torch

from mixture_experts_expert_histogram_amd import _lib


@pytest.fixture
def devices(monkeypatch):
    """Current device 0; device i's current stream is 100 + i; calls are recorded with the device they ran on."""
    state = types.SimpleNamespace(current=0, calls=[])

    class Guard:
        def __init__(self, d):
            self.to = getattr(d, "index", d)

        def __enter__(self):
            self.back, state.current = state.current, self.to

        def __exit__(self, *a):
            state.current = self.back

    def stream(d=None):
        return types.SimpleNamespace(cuda_stream=100 + (state.current if d is None else getattr(d, "index", d)))

    def record(*args):
        state.calls.append((state.current,) + tuple(getattr(a, "value", a) for a in args))
        return _lib.MOE_OK

    monkeypatch.setattr(torch.cuda, "current_device", lambda: state.current)
    monkeypatch.setattr(torch.cuda, "device", Guard)
    monkeypatch.setattr(torch.cuda, "current_stream", stream)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: 100 + i, raising=False)
    monkeypatch.setattr(_lib, "library", lambda: types.SimpleNamespace(moe_check_device_status=record))
    state.record = record
    return state


def buffer_on(index):
    return types.SimpleNamespace(device=types.SimpleNamespace(index=index, type="cuda"), is_cuda=True, data_ptr=lambda: 4096)


@pytest.mark.parametrize("index", [0, 1, 3])
def test_status_waits_for_the_workspace_device(devices, index):
    assert _lib.check_device_status(buffer_on(index)) == _lib.MOE_OK
    assert devices.calls == [(index, 4096, 100 + index)]
    assert devices.current == 0


@pytest.mark.parametrize("index", [0, 1, 3])
def test_serving_calls_run_on_their_device(devices, index):
    _lib._launch(buffer_on(index).device, "name", devices.record, 7)
    assert devices.calls == [(index, 7, 100 + index)]
    assert devices.current == 0
