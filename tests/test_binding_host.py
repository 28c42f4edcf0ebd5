"""The Python binding's use of torch, on the host."""
import types

import pytest

import skinny_gemv_gb300 as sg

torch = pytest.importorskip("torch")


@pytest.mark.parametrize("missing", [["_cuda_getDevice"], ["_cuda_getCurrentRawStream"],
                                     ["_cuda_getDevice", "_cuda_getCurrentRawStream"]])
def test_a_torch_without_the_private_names_is_enough(monkeypatch, missing):
    for name in ("_cuda_getDevice", "_cuda_getCurrentRawStream"):
        if name in missing:
            monkeypatch.delattr(torch._C, name, raising=False)
        else:
            monkeypatch.setattr(torch._C, name, (lambda *a: 3) if name == "_cuda_getDevice" else lambda d: 1000 + d,
                                raising=False)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d=None: types.SimpleNamespace(cuda_stream=1000 + d))
    for name in ("_torch_module", "_bf16", "_i32", "_u8", "_f32", "_get_device", "_raw_stream"):
        monkeypatch.setattr(sg, name, None)
    assert sg._torch() is torch
    assert sg._stream_handle(None) == 1003
    assert sg._stream_handle(7) == 7 and sg._stream_handle(types.SimpleNamespace(cuda_stream=9)) == 9
