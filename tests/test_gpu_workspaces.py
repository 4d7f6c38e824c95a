"""One workspace under all calls of a loop: fewer tokens, batches that shrink."""
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


def test_attention_of_batches_that_shrink():
    """Decoding with one buffer while sequences end: the results of calls with workspaces of their own."""
    H, Hq, D, page, n = 8, 40, 128, 64, 300
    most = 40
    g = torch.Generator(device="cuda").manual_seed(3)
    cache = B.kv_cache(n * 2, page, H, D)
    pages = torch.full((n, most), -1, dtype=torch.int32, device="cuda")
    pages[:, :2] = torch.randperm(n * 2, device="cuda", generator=g).to(torch.int32).view(n, 2)
    pages[:3, 2:] = pages[3:3 + 3 * 19, :2].reshape(3, 38)      # three long sequences share the others' pages
    lens = torch.full((n,), 128, dtype=torch.int32, device="cuda")
    K, V = (torch.randn(128 * n, H, D, device="cuda", generator=g).bfloat16() for _ in range(2))
    q_all = torch.arange(n + 1, dtype=torch.int32, device="cuda")
    B.w4a4_kv_append(K, V, B.kv_batch(q_all * 128, lens, pages, max_rows=128), cache)
    lens[:3] = most * page - 5
    size = B.w4a4_kv_attention_workspace_most(cache)
    ws = torch.full((size + 512,), 255, dtype=torch.uint8, device="cuda")
    Q = torch.randn(n, Hq, D, device="cuda", generator=g).bfloat16()
    sizes = []
    for m in (300, 200, 130, 64, 20, 3, 1):
        b = B.kv_batch(q_all[:m + 1], lens[:m], pages[:m], max_rows=1)
        O, P = torch.empty_like(Q[:m]), torch.empty_like(Q[:m])
        sizes.append(B.w4a4_kv_attention_workspace_size(m, b, Hq, cache))
        B.w4a4_kv_attention(Q[:m], b, cache, O, ws[:size])
        B.w4a4_kv_attention(Q[:m], b, cache, P, B.alloc_workspace_kv(m, b, Hq, cache))
        assert torch.equal(O, P) and not bool(torch.isnan(O).any()), m
    assert any(x < y for x, y in zip(sizes, sizes[1:])), sizes
    assert bool((ws[size:] == 255).all())


def test_a_batch_without_sequences():
    """Through the binding, whose empty tensors have no address: nothing is read or written."""
    cache = B.kv_cache(3, 16, 2, 64)
    cache.data.fill_(9)
    i32 = dict(dtype=torch.int32, device="cuda")
    b = B.kv_batch(torch.zeros(1, **i32), torch.zeros(0, **i32), torch.zeros(0, 4, **i32), max_rows=1)
    K = torch.ones(5, 2, 64, device="cuda")
    O, k = torch.full((5, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda"), torch.full((5, 2, 64), 7.0, device="cuda")
    B.w4a4_kv_append(K, K, b, cache)
    B.w4a4_kv_read(b, cache, k, k.clone())
    B.w4a4_kv_attention(torch.ones(5, 4, 64, device="cuda"), b, cache, O, B.alloc_workspace_kv(5, b, 4, cache))
    torch.cuda.synchronize()
    assert bool((cache.data == 9).all()) and bool((O == 7).all()) and bool((k == 7).all())
