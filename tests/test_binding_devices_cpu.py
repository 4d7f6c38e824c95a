"""Weights that stand on another device than the tensors are refused before the library is called: its kernels would
read addresses of that device.  The library and the current device are stand-ins; nothing reaches a GPU."""
import pytest
import torch

from bit_quantized_dit_amd import w4a4 as B

CALLS = {
    "w4a4_int8_linear": lambda p: B.w4a4_int8_linear(torch.zeros(3, 40), p, torch.zeros(3, 20), torch.zeros(512, dtype=torch.uint8)),
    "w4a4_int8_quantize_activations": lambda p: B.w4a4_int8_quantize_activations(torch.zeros(3, 40), p, torch.zeros(512, dtype=torch.uint8)),
    "w4a4_int8_gemm_prequantized": lambda p: B.w4a4_int8_gemm_prequantized(torch.zeros(512, dtype=torch.uint8), 3, p, torch.zeros(3, 20)),
}


@pytest.mark.parametrize("fn", CALLS)
def test_int8_weights_on_another_device(fn, monkeypatch):
    called = []

    class Library:
        def __getattr__(self, name):
            return lambda *a: called.append(name) or 0
    blob = torch.zeros(4096, dtype=torch.uint8)
    packed = B.PackedInt8(blob, B.W4A4Int8Packed(40, 20, 128, 32, blob.data_ptr(), blob.data_ptr()))
    monkeypatch.setattr(B, "lib", lambda: Library())
    monkeypatch.setattr(B, "_stream_on", lambda *a: None)
    monkeypatch.setattr(B, "_here", lambda t, name: t.get_device())      # as if the CPU were the current device
    CALLS[fn](packed)
    assert called == [fn]
    called.clear()
    monkeypatch.setattr(B, "_here", lambda t, name: 0)
    monkeypatch.setattr(B, "_buffer", lambda *a: None)
    monkeypatch.setattr(torch.Tensor, "get_device", lambda t: 0 if t is not blob else -1)
    with pytest.raises(ValueError, match="packed weights"):
        CALLS[fn](packed)
    assert called == []
