"""Sizes of workspaces over the shapes that a serving loop meets: what a buffer for the largest call has to hold.  No
call here reaches the GPU."""
import ctypes

import pytest

from bit_quantized_dit_amd import w4a4 as B

FAKE = 0x100000     # an aligned address that host-side logic never reads


@pytest.fixture(scope="module")
def L():
    import os
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
