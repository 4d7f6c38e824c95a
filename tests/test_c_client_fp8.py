"""The FP8 layer and the mixture-of-experts layer from plain C: tests/c/w4a4_fp8_client.c (C99,
hipMalloc'd buffers) agrees with the binding on the descriptors' sizes and, on the GPU, on every bit
of both outputs."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

from bit_quantized_dit_amd import w4a4 as B
from tests import test_c_client as C

SRC = os.path.join(C.ROOT, "tests", "c", "w4a4_fp8_client.c")
CLIENT = os.path.join(C.OUT_DIR, "w4a4_fp8_client")


def build_client(monkeypatch) -> str:
    monkeypatch.setattr(C, "SRC", SRC)
    monkeypatch.setattr(C, "CLIENT", CLIENT)
    return C.build_client()


def test_descriptors_and_sizes(monkeypatch):
    out = subprocess.run([build_client(monkeypatch), "host"], check=True, capture_output=True, text=True).stdout
    vals = {k: int(v) for k, v in (line.split() for line in out.strip().split("\n"))}
    assert vals == {"packed": ctypes.sizeof(B.W4A4Fp8Packed), "ws_layout": ctypes.sizeof(B.W4A4Fp8WsLayout), "moe": ctypes.sizeof(B.W4A4Moe),
                    "moe_ws_layout": ctypes.sizeof(B.W4A4MoeWsLayout), "packed_size": B.w4a4_fp8_packed_size(3, 300, 200), "packed_size_none": 1}


@pytest.mark.gpu
def test_outputs_match_the_binding(monkeypatch):
    import torch

    client = build_client(monkeypatch)
    T, d, f, E, k = 5, 300, 70, 6, 2
    rng = np.random.default_rng(3)
    X, router, gate, up, down, wo = (rng.standard_normal(s).astype(np.float32) * c for s, c in
                                     [((T, d), 1), ((E, d), 0.1), ((E, f, d), 0.05), ((E, f, d), 0.05), ((E, d, f), 0.05), ((d, d), 0.05)])
    fin, fout = os.path.join(C.OUT_DIR, "fp8_client_in.bin"), os.path.join(C.OUT_DIR, "fp8_client_out.bin")
    with open(fin, "wb") as h:
        h.write(np.array([T, d, f, E, k], dtype=np.int64).tobytes() + b"".join(np.ascontiguousarray(a, np.float32).tobytes() for a in
                                                                               (X, router, gate, up, down, wo)))
    r = subprocess.run([client, "run", fin, fout], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stderr
    got = np.fromfile(fout, np.float32).reshape(2, T, d)
    x, *w = (torch.from_numpy(np.ascontiguousarray(a, np.float32)).cuda() for a in (X, router, gate, up, down, wo))
    p = [B.w4a4_fp8_pack_weights(a) for a in w[1:]]
    Y = torch.empty(2, T, d, device="cuda")
    B.w4a4_fp8_linear(x, p[3], Y[0], B.alloc_workspace_fp8(T, p[3]))
    layer = B.moe_layer(w[0], p[0], p[1], p[2], k)
    B.w4a4_moe_forward(x, layer, Y[1], B.alloc_workspace_moe(T, layer))
    assert np.array_equal(got.view(np.uint32), Y.cpu().numpy().view(np.uint32))
