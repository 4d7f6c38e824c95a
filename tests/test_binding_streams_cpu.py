"""Buffers that the binding allocates and a call writes on a given stream: that stream waits for
the one they were allocated on, and the allocator hears of it.  The library and the streams are
stand-ins; nothing reaches a GPU."""
import ctypes

import numpy as np
import pytest
import torch

from bit_quantized_dit_amd import w4a4 as B


class Stream:
    def __init__(self, log, name):
        self.log, self.name, self.cuda_stream = log, name, 0x1000 + len(name)

    def wait_stream(self, other):
        self.log.append(("wait", self.name, other.name))


class Library:
    """Every entry point answers OK and notes its call; size queries say 512 bytes."""

    def __init__(self, log):
        self.log = log

    def __getattr__(self, fn):
        def call(*args):
            self.log.append(("call", fn))
            if fn.endswith("_size"):
                args[-1]._obj.value = 512
            return 0
        return call


CALLS = {
    "w4a4_fp8_pack_weights": lambda s: B.w4a4_fp8_pack_weights(torch.zeros(20, 40), stream=s),
    "w4a4_fp8_pack_codes": lambda s: B.w4a4_fp8_pack_codes(torch.zeros(20, 40, dtype=torch.uint8), torch.zeros(1, 1), stream=s),
    "w4a4_pack_weights": lambda s: B.w4a4_pack_weights(torch.zeros(20, 40), np.ones(40), np.zeros(0), 0, stream=s),
    "w4a4_pack_weights_dyn": lambda s: B.w4a4_pack_weights_dyn(torch.zeros(20, 40), np.ones(40), 2, 0, stream=s),
    "w4a4_column_absmax": lambda s: B.w4a4_column_absmax(torch.zeros(20, 40), stream=s),
    "w4a4_search_alpha_k": lambda s: B.w4a4_search_alpha_k(torch.zeros(20, 40), torch.zeros(20, 40), [0.5], [1], 0, stream=s),
}


@pytest.mark.parametrize("fn", CALLS)
def test_other_stream_waits_and_is_recorded(fn, monkeypatch):
    log = []
    current, other = Stream(log, "current"), Stream(log, "other")
    monkeypatch.setattr(B, "lib", lambda: Library(log))
    monkeypatch.setattr(B, "_dev", lambda *a: None)
    monkeypatch.setattr(B, "_raw_stream", None)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: current)
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: log.append(("record", s.name)))
    CALLS[fn](other)
    at = log.index(("call", fn))
    assert log.index(("wait", "other", "current")) < at and ("record", "other") in log
    for same in (None, current):
        log.clear()
        CALLS[fn](same)
        assert [x[0] for x in log if x[0] != "call"] == []
