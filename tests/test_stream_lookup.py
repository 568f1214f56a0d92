"""The lookup of the current stream's address, with and without torch's private
function for it."""
import importlib.util
import os
from types import SimpleNamespace

import pytest
import torch

import combine_moonep_plan_gb300 as pkg


def _fresh_api():
    path = os.path.join(os.path.dirname(pkg.__file__), "api.py")
    spec = importlib.util.spec_from_file_location(pkg.__name__ + "._api_copy", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def test_without_the_private_function(monkeypatch):
    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: SimpleNamespace(cuda_stream=4711))
    assert _fresh_api()._stream() == 4711


def test_with_it(monkeypatch):
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 100 + d, raising=False)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    assert _fresh_api()._stream() == 103


@pytest.mark.gpu
def test_on_a_side_stream():
    from combine_moonep_plan_gb300 import api
    side = torch.cuda.Stream()
    assert api._stream() == torch.cuda.current_stream().cuda_stream
    with torch.cuda.stream(side):
        assert api._stream() == side.cuda_stream
