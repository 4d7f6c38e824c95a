"""Sizes of workspaces over the shapes that a serving loop meets: what a buffer for the largest call has to hold; limits
as the header states them; batches without sequences.  No call here reaches the GPU."""
import ctypes
import os
import re
from types import SimpleNamespace

import pytest

from bit_quantized_dit_amd import w4a4 as B

FAKE = 0x100000     # an aligned address that host-side logic never reads


def _header(name):
    with open(os.path.join(os.path.dirname(__file__), "..", "include", "w4a4.h")) as f:
        return re.search(rf"define {name} (.*)", f.read()).group(1)


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(B.LIB_PATH):
        from bit_quantized_dit_amd import build
        build.build_library()
    return B.lib()


def _int8(d_in, d_out):
    return B.W4A4Int8Packed(d_in, d_out, -(-d_in // 128) * 128, -(-d_out // 16) * 16, FAKE, FAKE)


@pytest.mark.parametrize("d_in,d_out", [(5120, 5120), (5120, 13824), (13824, 5120), (4999, 1111), (13824, 512), (40000, 64), (20000, 48), (300, 200),
                                        (1100, 40), (2048, 2048), (131072, 4096), (1000, 40000)])
def test_int8_workspace_serves_fewer_tokens(L, d_in, d_out):
    """The size does not fall as tokens are added, across every change of plan."""
    d, out, before, at = _int8(d_in, d_out), B.W4A4Int8WsLayout(), 0, 0
    for T in list(range(1, 1200)) + list(range(1200, 20000, 37)) + list(range(20000, 140000, 1021)):
        assert L.w4a4_int8_workspace_layout(T, d, out) == 0
        assert out.total >= before, f"{T} tokens need {out.total} bytes, {at} need {before}"
        before, at = out.total, T
        codes = -(-T // 16) * 16 * d.k_pad + 4 * T
        assert codes <= out.total <= codes + (65 << 20)


def test_attention_workspaces_have_a_bound(L):
    """Sizes grow as batches shrink, but never past what the header names."""
    n = ctypes.c_size_t()

    def size(seqs, rows, max_pages, c, heads):
        b = B.W4A4KvBatch(seqs, rows, max_pages, FAKE, FAKE, FAKE)
        st = L.w4a4_kv_attention_workspace_size(1, b, c, heads, n)
        assert st in (0, 2)      # 2: more workgroups than a launch counts
        return n.value if st == 0 else 0
    assert _header(r"W4A4_KV_ATTENTION_WS_MOST\(d_pad\)") == "(((size_t)(d_pad) << 21) + ((size_t)1 << 23))"
    fell = False
    for D in (32, 64, 96, 128, 192, 256):
        for H in (1, 2, 8, 40):
            c = B.W4A4KvCache()
            assert L.w4a4_kv_cache_describe(1, 64, H, D, FAKE, B.w4a4_kv_cache_size(1, 64, H, D), c) == 0
            most = B.w4a4_kv_attention_workspace_most(SimpleNamespace(desc=c))
            assert most == (c.d_pad << 21) + (1 << 23)
            for ratio in (1, 5, 16, 64):
                for rows in (1, 2, 3, 4, 7, 16, 33, 64, 65, 200, 1000, 4096, 60000):
                    before = 0
                    for seqs in (1, 2, 3, 5, 13, 31, 64, 65, 100, 127, 128, 250, 500, 1000, 4095, 20000):
                        for max_pages in (4, 40, 900, 40000):
                            now = size(seqs, rows, max_pages, c, H * ratio)
                            assert now <= most, (D, H, ratio, rows, seqs, max_pages)
                        fell |= now < before
                        before = now
    assert fell


def test_int8_limits_are_the_headers(L):
    """Both sides of the largest number of tiles, at the widest layer, the most tokens, and ragged last tiles."""
    tiles = int(_header("W4A4_INT8_MAX_TILES").split()[0])
    size = ctypes.c_size_t()

    def status(T, d_out): return L.w4a4_int8_workspace_size(T, _int8(128, d_out), size)
    for d_out in (1 << 20, (1 << 20) - 255, 7936, 7937, 65536, 65537):
        nb = -(-d_out // 256)
        T = min(tiles // nb * 256, (1 << 26) - 16)
        assert status(T, d_out) == 0, (T, d_out)
        assert status(T + 1, d_out) == 2, (T, d_out)
    assert status((1 << 26) - 16, 7936) == 0 and status((1 << 26) - 16, 256 * (tiles >> 18) + 1) == 2


def test_batches_without_sequences(L):
    """Empty arrays have no address: such a batch is nothing to do, not an error."""
    c, n = B.W4A4KvCache(), ctypes.c_size_t(7)
    assert L.w4a4_kv_cache_describe(5, 16, 2, 72, FAKE, B.w4a4_kv_cache_size(5, 16, 2, 72), c) == 0
    rows = B.W4A4KvRows(FAKE, 288, 72, 1, 0)
    for at in ((None, None, None), (FAKE, None, None), (FAKE, FAKE, FAKE)):
        b = B.W4A4KvBatch(0, 4, 5, *at)
        assert L.w4a4_kv_attention_workspace_size(3, b, c, 4, n) == 0 and n.value == 0
        assert L.w4a4_kv_append(rows, rows, 3, b, c, None) == 0 and L.w4a4_kv_read(3, b, c, FAKE, FAKE, 0, None) == 0
        assert L.w4a4_kv_attention(rows, 3, b, c, 4, 0.1, 1, 0, FAKE, FAKE, 256, None) == 0
    b = B.W4A4KvBatch(1, 4, 5, FAKE, None, FAKE)
    assert L.w4a4_kv_append(rows, rows, 3, b, c, None) == 1
