"""The example that runs the FP8 layer and the mixture-of-experts layer together."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tokens", [1, 5, 40])
def test_fp8_experts(tokens):
    """bf16 results: each of the layer's two roundings (h, Y) and the residual's is at most 2^-8
    relative, so the norm is off by less than 2^-6."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "fp8_experts.py")
    spec = importlib.util.spec_from_file_location("fp8_experts", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    print(f"example tokens={tokens}", flush=True)
    err, us = mod.run(256, 200, 8, 2, tokens, steps=3)
    assert err < 2.0 ** -6 and us > 0
