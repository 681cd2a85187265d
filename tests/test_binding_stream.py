"""CPU: the binding's way to the current stream of a device, with and without torch's short one."""
import importlib.util
import os
import sys
import types

import torch

import w8a8_smoothquant_gemm_b200 as sq


def test_current_stream_without_the_short_way(monkeypatch):
    """torch._C is no public interface: where it lacks the call that gives a stream's handle, torch.cuda has it."""
    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
    monkeypatch.delattr(torch._C, "_cuda_getDevice", raising=False)
    asked = []

    def current_stream(device=None):
        asked.append(device)
        return types.SimpleNamespace(cuda_stream=0x70)

    monkeypatch.setattr(torch.cuda, "current_stream", current_stream)
    spec = importlib.util.spec_from_file_location("binding_copy", sq.__file__,
                                                  submodule_search_locations=[os.path.dirname(sq.__file__)])
    copy = importlib.util.module_from_spec(spec)
    monkeypatch.setitem(sys.modules, "binding_copy", copy)
    spec.loader.exec_module(copy)
    assert copy._raw_stream(3) == 0x70 and asked == [3]
    assert copy._current_device is torch.cuda.current_device
