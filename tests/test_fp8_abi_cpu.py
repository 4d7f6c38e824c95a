"""Host half of the FP8 layer and the mixture-of-experts layer (size queries, layouts,
refusals), and the pins of their 64-bit forms.  No call here reaches the GPU."""
import ctypes

import numpy as np
import pytest
import torch

from bit_quantized_dit_amd import w4a4 as B
from tests import fp8_ref as R

FAKE = 0x100000     # an aligned address that host-side logic never reads


@pytest.fixture(scope="module")
def L():
    import os
    if not os.path.exists(B.LIB_PATH):
        from bit_quantized_dit_amd import build
        build.build_library()
    return B.lib()


def _packed(n_mat=1, d_in=300, d_out=200, kind=0):
    d = B.W4A4Fp8Packed()
    d.n_mat, d.d_in, d.d_out, d.scale_kind = n_mat, d_in, d_out, kind
    d.k_pad, d.n_pad = -(-d_in // 128) * 128, -(-d_out // 16) * 16
    d.codes = d.scales = FAKE
    return d


def _moe(E=8, d=300, f=100, k=2, act=0):
    m = B.W4A4Moe()
    m.gate, m.up, m.down = _packed(E, d, f), _packed(E, d, f), _packed(E, f, d)
    m.router, m.router_dtype, m.top_k, m.renormalize, m.activation = FAKE, 1, k, 1, act
    return m


def test_packed_size(L):
    assert B.w4a4_fp8_packed_size(1, 512, 1024) == 1024 * 512 + 256          # 8 x 4 scales
    assert B.w4a4_fp8_packed_size(3, 300, 200) == 3 * 208 * 384 + 256
    for args, code in [((0, 5, 5), 1), ((1, 0, 5), 1), ((1, 5, 0), 1), ((1, -3, 5), 1), ((1, (1 << 20) + 1, 5), 2), ((1, 5, (1 << 20) + 1), 2),
                       ((65536, 5, 5), 2), ((60000, 1 << 20, 1 << 20), 2)]:
        assert L.w4a4_fp8_packed_size(*args, ctypes.byref(ctypes.c_size_t())) == code, args
    assert L.w4a4_fp8_packed_size(1, 5, 5, None) == 1


def test_workspace_layout(L):
    out = B.W4A4Fp8WsLayout()
    d = _packed()
    assert L.w4a4_fp8_workspace_layout(33, d, out) == 0
    assert out.a_q == 0 and out.a_s >= 48 * 384 and out.total >= out.a_s + 3 * 64 * 4 and out.total % 256 == 0
    n = ctypes.c_size_t()
    assert L.w4a4_fp8_workspace_size(0, d, n) == 0
    for change, code in [({"n_mat": 2}, 1), ({"k_pad": 300}, 1), ({"n_pad": 204}, 1), ({"scale_kind": 2}, 1), ({"codes": None}, 1),
                         ({"codes": FAKE + 8}, 3), ({"d_in": 0}, 1)]:
        d = _packed()
        for a, v in change.items():
            setattr(d, a, v)
        assert L.w4a4_fp8_workspace_layout(4, d, out) == code, change
    assert L.w4a4_fp8_workspace_layout(-1, _packed(), out) == 1
    assert L.w4a4_fp8_workspace_layout(1 << 40, _packed(), out) == 2
    assert L.w4a4_fp8_workspace_layout(4, None, out) == 1 and L.w4a4_fp8_workspace_layout(4, _packed(), None) == 1


def test_linear_refusals(L):
    d = _packed()
    n = ctypes.c_size_t()
    assert L.w4a4_fp8_workspace_size(4, d, n) == 0
    ok = [FAKE, 1, 4, d, FAKE, 0, FAKE, n.value, None]
    for i, v, code in [(0, None, 1), (0, FAKE + 4, 3), (1, 2, 1), (2, -1, 1), (3, None, 1), (4, None, 1), (4, FAKE + 2, 3), (5, 2, 1),
                       (6, None, 1), (6, FAKE + 1, 3), (7, n.value - 1, 2)]:
        bad = list(ok)
        bad[i] = v
        assert L.w4a4_fp8_linear(*bad) == code, (i, v)
    zero = list(ok)
    zero[2] = 0
    assert L.w4a4_fp8_linear(*zero) == 0
    assert L.w4a4_fp8_gemm_prequantized(FAKE, n.value, 4, d, None, 0, None) == 1
    assert L.w4a4_fp8_gemm_prequantized(FAKE, n.value, 4, d, FAKE, 7, None) == 1
    assert L.w4a4_fp8_quantize_activations(FAKE, 1, 4, d, FAKE, 0, None) == 2


def test_pack_refusals(L):
    d, n = B.W4A4Fp8Packed(), B.w4a4_fp8_packed_size(1, 40, 20)
    for i, v, code in [(0, None, 1), (0, FAKE + 2, 3), (1, 5, 1), (2, 0, 1), (5, 9, 1), (6, None, 1), (6, FAKE + 4, 3), (7, n - 1, 2), (8, None, 1)]:
        bad = [FAKE, 0, 1, 40, 20, 0, FAKE, n, d, None]
        bad[i] = v
        assert L.w4a4_fp8_pack_weights(*bad) == code, (i, v)
    for i, v, code in [(0, None, 1), (1, None, 1), (1, FAKE + 1, 3), (5, 2, 1), (7, 0, 2)]:
        bad = [FAKE, FAKE, 1, 40, 20, 0, FAKE, n, d, None]
        bad[i] = v
        assert L.w4a4_fp8_pack_codes(*bad) == code, (i, v)
    assert d.codes is None      # a refused call leaves the descriptor alone


def test_moe_layout_and_refusals(L):
    out, n = B.W4A4MoeWsLayout(), ctypes.c_size_t()
    m = _moe()
    assert L.w4a4_moe_workspace_layout(5, m, out) == 0
    order = [getattr(out, f) for f, _ in B.W4A4MoeWsLayout._fields_]
    assert order == sorted(order) and out.total - out.h >= 10 * 128 * 2 and out.ids - out.xb >= 5 * 384 * 2
    assert L.w4a4_moe_workspace_size(128, m, n) == 0 and L.w4a4_moe_workspace_size(129, m, n) == 2
    assert L.w4a4_moe_workspace_size(-1, m, n) == 1 and L.w4a4_moe_workspace_size(4, None, n) == 1

    def broken(**kw):
        x = _moe()
        for a, v in kw.items():
            setattr(x, a, v)
        return L.w4a4_moe_workspace_size(4, x, n)
    assert broken(top_k=0) == 1 and broken(top_k=9) == 1 and broken(activation=2) == 1 and broken(router_dtype=3) == 1
    assert broken(router=None) == 1 and broken(router=FAKE + 4) == 3
    assert broken(down=_packed(8, 100, 301)) == 2 and broken(down=_packed(7, 100, 300)) == 2 and broken(gate=_packed(8, 300, 99)) == 2
    assert broken(gate=B.W4A4Fp8Packed()) == 1
    assert broken(gate=B.W4A4Fp8Packed(), activation=1) == 0          # not read without a gate
    wide = _moe(E=64, k=33)
    assert L.w4a4_moe_workspace_size(4, wide, n) == 2
    assert L.w4a4_moe_workspace_size(4, _moe(E=1025), n) == 2
    assert L.w4a4_moe_workspace_size(4, _moe(d=65537), n) == 2
    L.w4a4_moe_workspace_size(4, m, n)
    ok = [FAKE, 1, 4, m, FAKE, 0, FAKE, n.value, None]
    for i, v, code in [(0, None, 1), (0, FAKE + 4, 3), (1, 2, 1), (2, -1, 1), (2, 129, 2), (4, None, 1), (4, FAKE + 2, 3), (5, 2, 1), (6, None, 1),
                       (7, n.value - 1, 2)]:
        bad = list(ok)
        bad[i] = v
        assert L.w4a4_moe_forward(*bad) == code, (i, v)
    zero = list(ok)
    zero[2] = 0
    assert L.w4a4_moe_forward(*zero) == 0


def test_code_values_and_rounding():
    """The value table is torch's E4M3; encoding is nearest with ties to even."""
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(np.isnan(t), np.isnan(R.VALUE)) and np.array_equal(t[~np.isnan(t)], R.VALUE[~np.isnan(t)])
    grid = R.VALUE[:0x7F]
    mid = (grid[1:] + grid[:-1]) / 2
    x = np.concatenate([grid, mid, np.nextafter(mid, 1e9), np.nextafter(mid, -1e9)]).astype(np.float32)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(R.encode(x), want) and np.array_equal(R.encode(-x) ^ 0x80, want)


def test_scale_rule():
    a = np.float32([448, 449, 224, 225, 1, 0, 2.0 ** -100, 3.0e38, np.inf, np.nan])
    p = R.scale_of(a, 1)
    assert p[:5].tolist() == [1, 2, 0.5, 1, 2.0 ** -8] and (p[5:7] == 2.0 ** -60).all() and np.isnan(p[8:]).all()
    fin = a[:5].astype(np.float64)
    assert (fin <= 448 * p[:5].astype(np.float64)).all() and (fin > 224 * p[:5].astype(np.float64)).all()
    s = R.scale_of(a, 0)
    assert s[0] == 1 and s[5] == 2.0 ** -60 and s[2] == 0.5 and np.isnan(s[8:]).all()


def test_choice_of_experts():
    l = np.float32([[0, 0, 0, 0], [1, 3, 3, 2], [-np.inf, np.nan, 5, np.nan], [-0.0, 0.0, -1, np.inf]])
    assert R.topk(l, 3).tolist() == [[0, 1, 2], [1, 2, 3], [1, 3, 2], [3, 0, 1]]


def test_untile_inverts_the_packed_order():
    rows, k = 64, 256
    r, p = np.meshgrid(np.arange(rows), np.arange(k), indexing="ij")
    off = ((r // 16) * (k // 128) + p // 128) * 2048 + ((p // 64) % 2) * 1024 + ((p // 8) % 4) * 256 + (r % 16) * 16 + ((p // 32) % 2) * 8 + p % 8
    assert np.array_equal(np.sort(off.ravel()), np.arange(rows * k))
    val = ((r * 7 + p * 13) % 251).astype(np.uint8)
    raw = np.zeros(rows * k, np.uint8)
    raw[off.ravel()] = val.ravel()
    assert np.array_equal(B.untile_fp8(torch.from_numpy(raw), rows, k).numpy(), val)


def test_plans(L):
    """Partial sums in the workspace, by form of the product: none, tiles of 128 x 128 and 256 x 256
    whose last round is split, the few-token kernel's row tiles."""
    out = B.W4A4Fp8WsLayout()
    for T, d_in, d_out, tiles, floats in [(1, 5120, 13824, 0, 0), (64, 512, 1024, 0, 0), (1100, 400, 1501, 0, 0),
                                          (1000, 2300, 1003, 0, 0), (1050, 2300, 1003, 9 * 8 * 4, 128 * 128), (2100, 1100, 2090, 9 * 9 * 2, 256 * 256),
                                          (4096, 13824, 5120, 64 * 4, 256 * 256), (24, 13824, 5120, 160 * 3, 32 * 32),
                                          (50, 8200, 4111, 129 * 3, 64 * 32), (3, 16500, 41, 3 * 4, 16 * 16)]:
        assert L.w4a4_fp8_workspace_layout(T, _packed(1, d_in, d_out), out) == 0
        assert out.count - out.partial == tiles * floats * 4, (T, d_in, d_out)
        assert out.total - out.count == (2048 if T <= 64 and tiles else 0)
    assert L.w4a4_fp8_workspace_layout(0, _packed(1, 13824, 5120), out) == 0 and out.total == 0


def test_sizes_that_a_launch_cannot_count(L):
    """Refused with a status of their own before anything reaches the device."""
    out = B.W4A4Fp8WsLayout()
    assert L.w4a4_fp8_workspace_layout(1 << 30, _packed(1, 1, 256), out) == 0
    assert L.w4a4_fp8_workspace_layout(1 << 31, _packed(1, 1, 256), out) == 2
    assert L.w4a4_fp8_workspace_layout((1 << 33) + 1, _packed(1, 1, 1), out) == 2
    assert B.w4a4_fp8_packed_size(4096, 1 << 20, 16) == (1 << 36) + (1 << 27)
