"""Calls on tensors of a device that is not the current one (host only, the runtime's answers replaced): the
entry point runs with that device current, on the stream that is current there, and an error status of
it is raised after the former device is back."""

import pytest
import torch

import w4a16_dequant_gemm_amd as W4


class Runtime:
    def __init__(self, monkeypatch, current):
        self.current, self.calls = current, []
        monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: 1000 + i, raising=False)
        monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: self.current, raising=False)
        runtime = self

        class Guard:
            def __init__(self, device):
                self.index = torch.device(device).index

            def __enter__(self):
                self.before, runtime.current = runtime.current, self.index

            def __exit__(self, *exc):
                runtime.current = self.before
                return False
        monkeypatch.setattr(torch.cuda, "device", Guard)

    def entry(self, status):
        def fn(*args):
            self.calls.append((self.current, args))
            return status
        return fn


@pytest.mark.parametrize("current,mine", [(0, 0), (0, 1), (3, 1)])
def test_the_call_runs_on_its_tensors_device(monkeypatch, current, mine):
    rt = Runtime(monkeypatch, current)
    W4._call(rt.entry(W4.OK), "entry", torch.device("cuda", mine), "a", 7)
    assert rt.calls == [(mine, ("a", 7, 1000 + mine))] and rt.current == current


@pytest.mark.parametrize("current,mine", [(0, 0), (0, 1)])
def test_an_error_is_raised_with_the_former_device_current(monkeypatch, current, mine):
    rt = Runtime(monkeypatch, current)
    with pytest.raises(W4.W4A16Error):
        W4._call(rt.entry(-2), "entry", torch.device("cuda", mine))
    assert rt.calls == [(mine, (1000 + mine,))] and rt.current == current
