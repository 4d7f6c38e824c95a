"""The INT8 linear layer on the GPU against its 64-bit form: codes and scales bit for bit,
outputs within three binary32 roundings (the integer sums are exact), at the sizes and values where a path changes."""
import numpy as np
import pytest
import torch

from bit_quantized_dit_amd import w4a4 as B
from tests import kv_ref as R

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


def _x(T, d, dtype, seed, heavy=True):
    rng = np.random.default_rng(seed)
    x = (rng.standard_normal((T, d)) * 0.3).astype(np.float32)
    if heavy:
        x[:, rng.integers(0, d, max(1, d // 80))] *= 20
    return torch.from_numpy(x).to(dtype).float().numpy()


def _guarded(x, dtype, fill):
    buf = torch.full((x.size + 512,), fill, dtype=dtype, device="cuda")
    buf[256:256 + x.size] = torch.from_numpy(np.ascontiguousarray(x).ravel()).to(dtype).cuda()
    return buf, buf[256:256 + x.size].view(x.shape)


def _check(x, xt, w, yt, wt=F32):
    T, (n, d) = x.shape[0], w.shape
    print(f"int8 linear T={T} {d}->{n} x={xt} y={yt}", flush=True)
    _, X = _guarded(x, xt, float("nan"))
    _, W = _guarded(w, wt, float("nan"))
    layer = B.w4a4_int8_pack_weights(W)
    wq, wsc = R.int8_quantize(w)
    v = layer.views()
    assert np.array_equal(v["codes"].cpu().numpy(), wq)
    assert np.array_equal(v["scales"].cpu().numpy(), wsc, equal_nan=True)
    ws = torch.full((max(B.w4a4_int8_workspace_size(T, layer), 256) + 512,), 255, dtype=torch.uint8, device="cuda")
    buf, Y = _guarded(np.zeros((T, n), np.float32), yt, 7.0)
    B.w4a4_int8_quantize_activations(X, layer, ws[:-512])
    q, s = R.int8_quantize(x)
    a = B.workspace_int8_views(ws, T, layer)
    assert np.array_equal(a["A_q"].cpu().numpy()[:, :d], q) and not bool(a["A_q"][:, d:].any())
    assert np.array_equal(a["A_s"].cpu().numpy(), s, equal_nan=True)
    B.w4a4_int8_gemm_prequantized(ws[:-512], T, layer, Y)
    first = Y.clone()
    ws.fill_(255)
    Y.fill_(3.0)
    B.w4a4_int8_linear(X, layer, Y, ws[:-512])
    torch.cuda.synchronize()
    assert torch.equal(first.view(torch.int32 if yt == F32 else torch.int16), Y.view(torch.int32 if yt == F32 else torch.int16))
    assert bool((ws[-512:] == 255).all()) and bool((buf[:256] == 7).all()) and bool((buf[256 + T * n:] == 7).all())
    ref, tol = R.int8_product(q, s, wq, wsc)
    if yt == BF16:
        tol = tol + R.BF16_U * (np.abs(ref) + tol)
    y = Y.double().cpu().numpy()
    assert np.array_equal(np.isnan(y), np.isnan(ref))
    ok = ~np.isnan(ref)
    bad = np.abs(y - ref)[ok] > tol[ok]
    assert not bad.any(), f"{int(bad.sum())} of {bad.size} outside three roundings"
    return y


SHAPES = [(1, 1, 1), (1, 128, 16), (2, 127, 17), (5, 129, 33), (16, 256, 128), (17, 300, 257), (31, 1100, 40),
          (33, 640, 96), (64, 2176, 130), (65, 384, 129), (100, 1000, 300), (129, 128, 128), (257, 512, 1024),
          (300, 333, 1111), (1, 40000, 64), (40, 20000, 48), (20, 13824, 2500), (3, 5200, 24)]


@pytest.mark.parametrize("T,d,n", SHAPES)
def test_shapes(T, d, n):
    w = (np.random.default_rng(T * 7 + d).standard_normal((n, d)) * 0.02).astype(np.float32)
    _check(_x(T, d, BF16, 1), BF16, w, F32)
    _check(_x(T, d, F32, 2), F32, w, BF16)
    wb = torch.from_numpy(w).bfloat16().float().numpy()
    _check(_x(T, d, F32, 2), F32, wb, F32, BF16)


@pytest.mark.parametrize("T,d,n,yt", [(4001, 200, 3211, F32), (4001, 200, 3211, BF16), (2048, 256, 6144, BF16), (2100, 2500, 2600, F32),
                                      (1100, 1200, 1030, BF16), (5000, 5120, 40, F32)])
def test_large_tiles(T, d, n, yt):
    w = (np.random.default_rng(5).standard_normal((n, d)) * 0.02).astype(np.float32)
    _check(_x(T, d, BF16, 3), BF16, w, yt)


@pytest.mark.parametrize("T", [3, 40, 200, 1500])
def test_special_values(T):
    """Zero rows, rows whose scale sits at its floor, the largest finite values, ties; a NaN or an
    infinity makes its own row NaN and no other, in a weight row its own column."""
    d, n = 400, 144
    x = _x(T, d, F32, 11)
    w = (np.random.default_rng(12).standard_normal((n, d)) * 0.02).astype(np.float32)
    x[0] = 0
    x[0, 3] = -0.0
    x[1] = 0
    x[1, :9] = [127, 0.5, 1.5, 2.5, -0.5, -1.5, 126.5, -126.5, 0.49999997]
    x[2] = np.float32(1e-42)
    y = _check(x, F32, w, F32)
    assert np.isfinite(y).all() and not y[0].any()
    for bad in (np.nan, np.inf, -np.inf):
        z = x.copy()
        z[T // 2, 300] = bad
        y2 = _check(z, F32, w, F32)
        keep = np.arange(T) != T // 2
        assert np.isnan(y2[T // 2]).all() and np.array_equal(y2[keep], y[keep])
    w2 = w.copy()
    w2[17, 5] = np.nan
    y2 = _check(x, F32, w2, F32)
    assert np.isnan(y2[:, 17]).all() and np.array_equal(np.delete(y2, 17, 1), np.delete(y, 17, 1))
    big = x.copy()
    big[0, 5] = 3.0e38
    _check(big, F32, w, F32)


@pytest.mark.parametrize("T,d,n", [(5, 131072, 32), (300, 131072, 160), (3, 200, 70)])
def test_checkpoint_codes_and_the_largest_sums(T, d, n):
    """Codes of a checkpoint taken as they are, -128 included; sums next to 2^31."""
    g = torch.Generator(device="cuda").manual_seed(1)
    codes = torch.randint(-128, 128, (n, d), dtype=torch.int8, device="cuda", generator=g)
    codes[0], codes[1] = -128, 127
    scales = torch.rand(n, device="cuda", generator=g) + 0.5
    layer = B.w4a4_int8_pack_codes(codes, scales)
    assert torch.equal(layer.views()["codes"], codes) and torch.equal(layer.views()["scales"], scales)
    X = torch.full((T, d), 1.0, device="cuda")
    X[1::2] = -1.0
    Y = torch.empty(T, n, device="cuda")
    B.w4a4_int8_linear(X, layer, Y, B.alloc_workspace_int8(T, layer))
    s = float(np.float32(1) / np.float32(127))
    ref = (X.sign() * 127).double() @ codes.double().t() * (s * scales.double())[None]
    assert bool(((Y.double() - ref).abs() <= 3.01 * R.F32_U * ref.abs()).all())


def test_one_quantization_for_several_layers():
    """The codes of one call serve layers of other widths, in a workspace large enough for each."""
    T, d = 40, 5000
    X = torch.randn(T, d, device="cuda")
    layers = [B.w4a4_int8_pack_weights(torch.randn(n, d, device="cuda")) for n in (600, 48, 3000)]
    ws = torch.full((max(B.w4a4_int8_workspace_size(T, p) for p in layers),), 255, dtype=torch.uint8, device="cuda")
    B.w4a4_int8_quantize_activations(X, layers[0], ws)
    for p in layers:
        a, b = torch.empty(T, p.d_out, device="cuda"), torch.empty(T, p.d_out, device="cuda")
        B.w4a4_int8_gemm_prequantized(ws, T, p, a)
        B.w4a4_int8_linear(X, p, b, B.alloc_workspace_int8(T, p))
        assert torch.equal(a, b)


@pytest.mark.parametrize("T,d,n", [(1, 5120, 640), (24, 13824, 512), (300, 1500, 1200), (4096, 1024, 2304)])
def test_graph_and_streams(T, d, n):
    """Captured and replayed with new inputs and eager work between; the same on another stream."""
    layer = B.w4a4_int8_pack_weights(torch.randn(n, d, device="cuda"))
    X = torch.randn(T, d, device="cuda").bfloat16()
    ws, ws2 = B.alloc_workspace_int8(T, layer), B.alloc_workspace_int8(T, layer)
    Y, Z = torch.empty(T, n, device="cuda"), torch.empty(T, n, device="cuda")
    B.w4a4_int8_linear(X, layer, Y, ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        B.w4a4_int8_linear(X, layer, Y, ws)
    st = torch.cuda.Stream()
    for i in range(4):
        X.normal_()
        g.replay()
        torch.cuda.synchronize()
        B.w4a4_int8_linear(X, layer, Z, ws2, stream=st)
        st.synchronize()
        assert torch.equal(Y, Z), i


def test_refusals():
    layer = B.w4a4_int8_pack_weights(torch.zeros(20, 40, device="cuda"))
    X, Y, ws = torch.zeros(4, 40, device="cuda"), torch.zeros(4, 20, device="cuda"), B.alloc_workspace_int8(4, layer)
    with pytest.raises(TypeError):
        B.w4a4_int8_linear(X.half(), layer, Y, ws)
    with pytest.raises(TypeError):
        B.w4a4_int8_linear(X, layer, Y.half(), ws)
    with pytest.raises(ValueError):
        B.w4a4_int8_linear(X[:, :39].contiguous(), layer, Y, ws)
    with pytest.raises(ValueError):
        B.w4a4_int8_linear(X, layer, Y[:3], ws)
    with pytest.raises(ValueError):
        B.w4a4_int8_linear(X.t().contiguous().t(), layer, Y, ws)
    with pytest.raises(B.W4A4Error):
        B.w4a4_int8_linear(X, layer, Y, ws[:64])
    with pytest.raises(TypeError):
        B.w4a4_int8_pack_codes(torch.zeros(4, 4, dtype=torch.uint8, device="cuda"), torch.ones(4, device="cuda"))
    with pytest.raises(ValueError):
        B.w4a4_int8_pack_codes(torch.zeros(4, 4, dtype=torch.int8, device="cuda"), torch.ones(3, device="cuda"))
    B.w4a4_int8_linear(X[:0], layer, Y[:0], ws)
