"""The INT8 layer, the 4-bit key/value cache and attention over it from plain C: tests/c/w4a4_kv_client.c
(C99, hipMalloc'd buffers) agrees with the binding on the descriptors' sizes and, on the GPU, on every
bit of the outputs."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

from bit_quantized_dit_amd import w4a4 as B
from tests import test_c_client as C

SRC = os.path.join(C.ROOT, "tests", "c", "w4a4_kv_client.c")
CLIENT = os.path.join(C.OUT_DIR, "w4a4_kv_client")


def build_client(monkeypatch) -> str:
    monkeypatch.setattr(C, "SRC", SRC)
    monkeypatch.setattr(C, "CLIENT", CLIENT)
    return C.build_client()


def test_descriptors_and_sizes(monkeypatch):
    out = subprocess.run([build_client(monkeypatch), "host"], check=True, capture_output=True, text=True).stdout
    vals = {k: int(v) for k, v in (line.split() for line in out.strip().split("\n"))}
    assert vals == {"int8_packed": ctypes.sizeof(B.W4A4Int8Packed), "int8_ws_layout": ctypes.sizeof(B.W4A4Int8WsLayout),
                    "cache": ctypes.sizeof(B.W4A4KvCache), "batch": ctypes.sizeof(B.W4A4KvBatch), "rows": ctypes.sizeof(B.W4A4KvRows),
                    "int8_packed_size": B.w4a4_int8_packed_size(300, 200), "cache_size": B.w4a4_kv_cache_size(7, 32, 3, 72), "cache_size_none": 1}


@pytest.mark.gpu
@pytest.mark.parametrize("T", [5, 77])
def test_outputs_match_the_binding(monkeypatch, T):
    import torch

    client = build_client(monkeypatch)
    d, Hq, H, D = 100, 6, 2, 40
    wide = (Hq + 2 * H) * D
    rng = np.random.default_rng(5)
    X, W = rng.standard_normal((T, d)).astype(np.float32), (rng.standard_normal((wide, d)) * 0.2).astype(np.float32)
    fin, fout = os.path.join(C.OUT_DIR, "kv_client_in.bin"), os.path.join(C.OUT_DIR, "kv_client_out.bin")
    with open(fin, "wb") as h:
        h.write(np.array([T, d, Hq, H, D], dtype=np.int64).tobytes() + X.tobytes() + W.tobytes())
    r = subprocess.run([client, "run", fin, fout], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stderr
    packed = B.w4a4_int8_pack_weights(torch.from_numpy(W).cuda())
    P = torch.empty(T, wide, device="cuda")
    B.w4a4_int8_linear(torch.from_numpy(X).cuda(), packed, P, B.alloc_workspace_int8(T, packed))
    n = -(-T // 16)
    cache = B.kv_cache(n, 16, H, D)
    batch = B.kv_batch(*(torch.tensor(v, dtype=torch.int32, device="cuda") for v in ([0, T], [T], [list(range(n))[::-1]])), T)
    q, k, v = (t.view(T, -1, D) for t in P.split([Hq * D, H * D, H * D], 1))
    B.w4a4_kv_append(k, v, batch, cache)
    O = torch.empty(T, Hq, D, dtype=torch.bfloat16, device="cuda")
    B.w4a4_kv_attention(q, batch, cache, O, B.alloc_workspace_kv(T, batch, Hq, cache), scale=0.125)
    K, V = torch.empty(T, H, D, device="cuda"), torch.empty(T, H, D, device="cuda")
    B.w4a4_kv_read(batch, cache, K, V)
    want = b"".join(t.cpu().contiguous().view(torch.uint8).numpy().tobytes() for t in (P, O, K, V))
    with open(fout, "rb") as h:
        assert h.read() == want
