"""One workspace, for the largest call of a loop, under calls of fewer tokens."""
import pytest
import torch

from bit_quantized_dit_amd import w4a4 as B

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d,n", [(5120, 5120), (13824, 512), (4999, 1111)])
def test_int8_calls_of_fewer_tokens(d, n):
    layer = B.w4a4_int8_pack_weights(torch.randn(n, d, device="cuda"))
    most = 2048
    size = B.w4a4_int8_workspace_size(most, layer)
    ws = torch.full((size + 512,), 255, dtype=torch.uint8, device="cuda")
    X = torch.randn(most, d, device="cuda").bfloat16()
    for T in (2048, 1024, 1000, 600, 333, 64, 40, 24, 7, 1, 2048):
        Y, Z = torch.empty(T, n, device="cuda"), torch.empty(T, n, device="cuda")
        B.w4a4_int8_linear(X[:T], layer, Y, ws[:size])
        B.w4a4_int8_linear(X[:T], layer, Z, B.alloc_workspace_int8(T, layer))
        assert torch.equal(Y, Z), T
        B.w4a4_int8_quantize_activations(X[:T], layer, ws[:size])
        Y.zero_()
        B.w4a4_int8_gemm_prequantized(ws[:size], T, layer, Y)
        assert torch.equal(Y, Z), T
    assert bool((ws[size:] == 255).all())
