"""Host half of the INT8 layer, the 4-bit key/value cache and attention over it (sizes, layouts,
refusals), and the pins of their 64-bit forms.  No call here reaches the GPU."""
import ctypes
import math

import numpy as np
import pytest
import torch

from bit_quantized_dit_amd import w4a4 as B
from tests import kv_ref as R

FAKE = 0x100000     # an aligned address that host-side logic never reads


@pytest.fixture(scope="module")
def L():
    import os
    if not os.path.exists(B.LIB_PATH):
        from bit_quantized_dit_amd import build
        build.build_library()
    return B.lib()


def _packed(d_in=300, d_out=200):
    return B.W4A4Int8Packed(d_in, d_out, -(-d_in // 128) * 128, -(-d_out // 16) * 16, FAKE, FAKE)


def test_int8_sizes(L):
    assert B.w4a4_int8_packed_size(512, 1024) == 1024 * 512 + 4096
    assert B.w4a4_int8_packed_size(300, 200) == 208 * 384 + 1024
    for args, code in [((0, 5), 1), ((5, 0), 1), ((-3, 5), 1), ((131073, 5), 2), ((5, (1 << 20) + 1), 2), ((131072, 1 << 20), 0)]:
        assert L.w4a4_int8_packed_size(*args, ctypes.byref(ctypes.c_size_t())) == code, args
    assert L.w4a4_int8_packed_size(5, 5, None) == 1
    out = B.W4A4Int8WsLayout()
    assert L.w4a4_int8_workspace_layout(33, _packed(), out) == 0
    assert out.a_q == 0 and out.a_s >= 48 * 384 and out.partial >= out.a_s + 33 * 4 and out.total % 256 == 0
    for change, code in [({"k_pad": 300}, 1), ({"n_pad": 204}, 1), ({"codes": None}, 1), ({"scales": None}, 1), ({"codes": FAKE + 8}, 3),
                         ({"d_in": 0}, 1), ({"d_in": 1 << 18}, 2)]:
        d = _packed()
        for a, v in change.items():
            setattr(d, a, v)
        assert L.w4a4_int8_workspace_layout(4, d, out) == code, change
    assert L.w4a4_int8_workspace_layout(-1, _packed(), out) == 1 and L.w4a4_int8_workspace_layout((1 << 26) + 1, _packed(), out) == 2
    assert L.w4a4_int8_workspace_layout((1 << 26) - 15, _packed(), out) == 2 and L.w4a4_int8_workspace_layout((1 << 26) - 16, _packed(), out) == 0
    assert L.w4a4_int8_workspace_layout(4, None, out) == 1 and L.w4a4_int8_workspace_layout(4, _packed(), None) == 1


def test_int8_refusals(L):
    d, n = _packed(), ctypes.c_size_t()
    assert L.w4a4_int8_workspace_size(4, d, n) == 0
    ok = [FAKE, 1, 4, d, FAKE, 0, FAKE, n.value, None]
    for i, v, code in [(0, None, 1), (0, FAKE + 4, 3), (1, 2, 1), (2, -1, 1), (3, None, 1), (4, None, 1), (4, FAKE + 2, 3), (5, 2, 1),
                       (6, None, 1), (6, FAKE + 1, 3), (7, n.value - 1, 2)]:
        bad = list(ok)
        bad[i] = v
        assert L.w4a4_int8_linear(*bad) == code, (i, v)
    ok[2] = 0
    assert L.w4a4_int8_linear(*ok) == 0
    assert L.w4a4_int8_gemm_prequantized(FAKE, n.value, 4, d, None, 0, None) == 1
    assert L.w4a4_int8_gemm_prequantized(FAKE, n.value, 4, d, FAKE, 7, None) == 1
    assert L.w4a4_int8_quantize_activations(FAKE, 1, 4, d, FAKE, 0, None) == 2
    d, n = B.W4A4Int8Packed(), B.w4a4_int8_packed_size(40, 20)
    for i, v, code in [(0, None, 1), (0, FAKE + 2, 3), (1, 5, 1), (2, 0, 1), (4, None, 1), (4, FAKE + 4, 3), (5, n - 1, 2), (6, None, 1)]:
        bad = [FAKE, 0, 40, 20, FAKE, n, d, None]
        bad[i] = v
        assert L.w4a4_int8_pack_weights(*bad) == code, (i, v)
    for i, v, code in [(0, None, 1), (1, None, 1), (1, FAKE + 1, 3), (5, 0, 2)]:
        bad = [FAKE, FAKE, 40, 20, FAKE, n, d, None]
        bad[i] = v
        assert L.w4a4_int8_pack_codes(*bad) == code, (i, v)
    assert d.codes is None      # a refused call leaves the descriptor alone


def _cache(n_pages=5, page=16, H=2, D=72, data=FAKE):
    c = B.W4A4KvCache()
    n = B.w4a4_kv_cache_size(n_pages, page, H, D)
    assert B.lib().w4a4_kv_cache_describe(n_pages, page, H, D, data, n, c) == 0
    return c


def test_cache_size_and_descriptor(L):
    for D, block in [(1, 544), (32, 544), (33, 1088), (64, 1088), (72, 1664), (96, 1664), (100, 2176), (128, 2176), (129, 3328), (192, 3328),
                     (193, 4352), (256, 4352)]:
        assert B.w4a4_kv_cache_size(3, 48, 2, D) == 3 * 2 * 3 * block
        c = _cache(3, 48, 2, D)
        assert (c.n_pages, c.page_tokens, c.n_heads, c.head_dim, c.d_pad, c.block_bytes) == (3, 48, 2, D, R.d_pad(D), block)
    n = ctypes.c_size_t()
    for args, code in [((0, 16, 1, 64), 1), ((1, 0, 1, 64), 1), ((1, 24, 1, 64), 1), ((1, 16, 0, 64), 1), ((1, 16, 1, 0), 1), ((1, 16, 1, 257), 2),
                       ((1, 16, 4097, 64), 2), ((1 << 31, 16, 1, 64), 2), ((1, (1 << 20) + 16, 1, 64), 2), ((0x7FFFFFFF, 1 << 20, 4096, 256), 2)]:
        assert L.w4a4_kv_cache_size(*args, n) == code, args
    assert L.w4a4_kv_cache_size(1, 16, 1, 64, None) == 1
    c, size = B.W4A4KvCache(), B.w4a4_kv_cache_size(1, 16, 1, 64)
    for data, nbytes, out, code in [(None, size, c, 1), (FAKE + 8, size, c, 3), (FAKE, size - 1, c, 2), (FAKE, size, None, 1)]:
        assert L.w4a4_kv_cache_describe(1, 16, 1, 64, data, nbytes, out) == code
    assert c.data is None


def _batch(n=3, max_rows=4, max_pages=5):
    return B.W4A4KvBatch(n, max_rows, max_pages, FAKE, FAKE, FAKE)


def test_kv_refusals(L):
    rows = B.W4A4KvRows(FAKE, 288, 72, 1, 0)
    size = ctypes.c_size_t()
    ok = [rows, 7, _batch(), _cache(), 4, 0.1, 1, 0, FAKE, FAKE, 1 << 40, None]
    assert L.w4a4_kv_attention_workspace_size(7, _batch(max_pages=400), _cache(), 4, size) == 0 and size.value > 0

    def attention(i, v):
        bad = list(ok)
        bad[i] = v
        return L.w4a4_kv_attention(*bad)
    for i, v, code in [(0, None, 1), (1, -1, 1), (1, (1 << 26) + 1, 2), (2, None, 1), (3, None, 1), (4, 0, 1), (4, 3, 1), (4, 4098, 2), (5, 0.0, 1),
                       (5, -1.0, 1), (5, math.nan, 1), (5, math.inf, 1), (5, 3e38, 1), (6, 2, 1), (7, -1, 1), (8, None, 1), (8, FAKE + 2, 3), (9, None, 1),
                       (9, FAKE + 4, 3)]:
        assert attention(i, v) == code, (i, v)
    bad = list(ok)
    bad[6], bad[7] = 0, 5
    assert L.w4a4_kv_attention(*bad) == 1      # a window without causal
    bad = list(ok)
    bad[2], bad[10] = _batch(max_pages=400), size.value - 1
    assert L.w4a4_kv_attention(*bad) == 2
    for field, v, code in [("data", None, 1), ("data", FAKE + 1, 3), ("dtype", 2, 1)]:
        r = B.W4A4KvRows(FAKE, 288, 72, 1, 0)
        setattr(r, field, v)
        assert attention(0, r) == code and L.w4a4_kv_append(r, rows, 7, _batch(), _cache(), None) == code
        assert L.w4a4_kv_append(rows, r, 7, _batch(), _cache(), None) == code
    r = B.W4A4KvRows(FAKE + 2, 288, 72, 0, 0)
    assert attention(0, r) == 3                # fp32 at a bf16's alignment
    assert L.w4a4_kv_append(rows, B.W4A4KvRows(FAKE, 288, 72, 0, 0), 7, _batch(), _cache(), None) == 1      # two types
    for field, v, code in [("n_seqs", -1, 1), ("n_seqs", 65536, 2), ("max_rows", -1, 1), ("max_rows", (1 << 26) + 1, 2), ("max_pages", 0, 1),
                           ("max_pages", 1 << 27, 2), ("q_start", None, 1), ("lens", None, 1), ("pages", None, 1), ("pages", FAKE + 2, 3)]:
        b = _batch()
        setattr(b, field, v)
        assert attention(2, b) == code, (field, v)
        assert L.w4a4_kv_append(rows, rows, 7, b, _cache(), None) == code and L.w4a4_kv_read(7, b, _cache(), FAKE, FAKE, 0, None) == code
    b = _batch(65535, 1 << 20)                 # more workgroups than a launch counts
    assert attention(2, b) == 2 and L.w4a4_kv_append(rows, rows, 7, b, _cache(), None) == 2
    for field, v, code in [("data", None, 1), ("data", FAKE + 8, 3), ("d_pad", 64, 1), ("block_bytes", 1088, 1), ("page_tokens", 20, 1), ("n_pages", 0, 1)]:
        c = _cache()
        setattr(c, field, v)
        assert attention(3, c) == code and L.w4a4_kv_read(7, _batch(), c, FAKE, FAKE, 0, None) == code, (field, v)
    for i, v, code in [(3, None, 1), (4, None, 1), (3, FAKE + 4, 3), (4, FAKE + 4, 3), (5, 2, 1)]:
        bad = [7, _batch(), _cache(), FAKE, FAKE, 0, None]
        bad[i] = v
        assert L.w4a4_kv_read(*bad) == code, (i, v)
    # nothing to do: no launch
    for n, b in [(0, _batch()), (7, _batch(n=0)), (7, _batch(max_rows=0))]:
        assert L.w4a4_kv_append(rows, rows, n, b, _cache(), None) == 0 and L.w4a4_kv_read(n, b, _cache(), FAKE, FAKE, 0, None) == 0
        assert L.w4a4_kv_attention(rows, n, b, _cache(), 4, 0.1, 1, 0, FAKE, FAKE, 1 << 40, None) == 0


def test_workspace_holds_what_a_plan_splits(L):
    """Long tables are cut into ranges, short ones, many row tiles and more sequences than fill the device are not;
    room for the ranges is bounded whatever the number of sequences."""
    n = ctypes.c_size_t()
    for batch, split in [(_batch(1, 1, 4000), True), (_batch(1, 1, 8), False), (_batch(1, 1 << 16, 40000), False), (_batch(1, 200, 40000), True)]:
        assert L.w4a4_kv_attention_workspace_size(9, batch, _cache(H=8, D=128), 8, n) == 0
        assert (n.value > 0) == split, (batch.n_seqs, batch.max_rows, batch.max_pages, n.value)
    for seqs in (64, 1000, 65535):
        assert L.w4a4_kv_attention_workspace_size(seqs, _batch(seqs, 1, 40000), _cache(H=8, D=128), 40, n) == 0
        assert n.value < 32 << 20 and (n.value > 0) == (seqs == 64)


def test_int8_form():
    x = np.float32([[127, 0.5, 1.5, 2.5, -0.5, -126.5], [0] * 6, [1, np.nan, 3, 4, 5, 6], [1e-30] * 6, [-3e38, 3e38, 1, 0, 0, 0]])
    q, s = R.int8_quantize(x)
    assert q[0].tolist() == [127, 0, 2, 2, 0, -126] and s[0] == 1 and s[1] == 2.0 ** -60 and not q[1].any()
    assert np.isnan(s[2]) and not q[2].any() and s[3] == 2.0 ** -60 and q[4].tolist() == [-127, 127, 0, 0, 0, 0]


def test_mxfp4_form():
    """The values are nearest in the scaled grid and the block layout covers every byte once."""
    rng = np.random.default_rng(0)
    x = (rng.standard_normal((300, 72)) * np.exp2(rng.integers(-20, 20, (300, 1)))).astype(np.float32)
    nib, sc, v = R.mxfp4(x)
    grid = np.concatenate([R.E2M1, -R.E2M1])
    p = np.zeros((300, 96))
    p[:, :72] = x
    s = np.exp2(sc.astype(np.float64) - 127).repeat(32, 1)
    amax = np.abs(p.reshape(300, 3, 32)).max(2)
    assert (np.exp2(sc - 127.0) * 4 <= amax).all() and (amax < np.exp2(sc - 127.0) * 8).all()
    best = np.abs(p[..., None] / s[..., None] - grid).min(-1)
    assert np.allclose(np.abs(p / s - grid[nib]), best) and np.array_equal((grid[nib] * s)[:, :72], v)
    for d in (20, 64, 80, 128, 160, 256):
        g = R.d_pad(d) // 32
        sg = g if g <= 2 else -(-g // 4) * 4
        seen = np.zeros(512 * g + 32 * sg, int)
        for b in range(len(seen)):
            raw = np.zeros(len(seen), np.uint8)
            raw[b] = 0xFF
            seen[b] = sum(int((a != 0).sum()) for a in R.decode_block(raw, d))
        assert (seen[:512 * g] == 2).all() and seen[512 * g:].sum() == 32 * g and seen.max() == 2


def test_attention_form():
    """Against torch's softmax, with rows that see nothing and values that are NaN."""
    g = torch.Generator().manual_seed(0)
    q, k, v = (torch.randn(n, 24, generator=g, dtype=torch.float64) for n in (5, 11, 11))
    lo, hi = np.array([0, 0, 3, 8, 4]), np.array([11, 5, 9, 8, 5])
    o, tol, var = R.attention(q, k, v, 0.3, lo, hi, True)
    for i in range(5):
        want = torch.softmax(0.3 * k[lo[i]:hi[i]] @ q[i], 0) @ v[lo[i]:hi[i]] if hi[i] > lo[i] else torch.zeros(24, dtype=torch.float64)
        assert torch.allclose(o[i], want, rtol=1e-12, atol=1e-14)
    assert bool((tol >= o.abs() * 2.0 ** -8).all()) and bool((var >= 0).all())
    v[6, 3] = math.nan
    o2, _, _ = R.attention(q, k, v, 0.3, lo, hi, True)
    assert torch.isnan(o2).nonzero().tolist() == [[0, 3], [2, 3]]
