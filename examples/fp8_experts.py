"""An FP8 projection and a mixture-of-experts layer of one transformer block, for a few tokens:

    A = X + X Wo^T          (w4a4_fp8_linear)
    Y = A + experts(A)      (w4a4_moe_forward)

captured into a HIP graph as a decoding loop would run it, and compared with the same formulas in
64 bits on the dequantized weights.  `python examples/fp8_experts.py` on an MI355X."""
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from bit_quantized_dit_amd import w4a4 as B


class Block:
    def __init__(self, d, f, n_experts, top_k, tokens, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def weights(*shape):
            return torch.randn(*shape, device="cuda", generator=g) * shape[-1] ** -0.5

        self.wo = B.w4a4_fp8_pack_weights(weights(d, d))
        mats = [B.w4a4_fp8_pack_weights(weights(n_experts, *s)) for s in ((f, d), (f, d), (d, f))]
        self.router = weights(n_experts, d).bfloat16()
        self.experts = B.moe_layer(self.router, *mats, top_k=top_k)
        self.X = torch.zeros(tokens, d, dtype=torch.bfloat16, device="cuda")
        self.A, self.Y = torch.empty_like(self.X), torch.empty_like(self.X)
        self.ws_o, self.ws_e = B.alloc_workspace_fp8(tokens, self.wo), B.alloc_workspace_moe(tokens, self.experts)
        self.mats = mats

    def forward(self):
        B.w4a4_fp8_linear(self.X, self.wo, self.A, self.ws_o)
        self.A += self.X
        B.w4a4_moe_forward(self.A, self.experts, self.Y, self.ws_e)
        self.Y += self.A
        return self.Y

    def exact(self):
        """Y in 64 bits from A as the projection left it (its own check is the codes' product)."""
        gate, up, down = (dequantize(m) for m in self.mats)
        a = self.A.double()
        p = torch.softmax(a @ self.router.double().t(), 1)
        w, ids = p.topk(self.experts.top_k, 1)
        w = w / w.sum(1, keepdim=True)
        y = a.clone()
        for t in range(a.shape[0]):
            for j, e in enumerate(ids[t].tolist()):
                y[t] += w[t, j] * (down[e] @ (torch.nn.functional.silu(gate[e] @ a[t]) * (up[e] @ a[t])))
        return y


def dequantize(m):
    v = m.views()
    c, s = v["codes"].view(torch.float8_e4m3fn).double(), v["scales"].double()
    return c * s.repeat_interleave(128, 1).repeat_interleave(128, 2)[:, :c.shape[1], :c.shape[2]]


def run(d, f, n_experts, top_k, tokens, steps=50):
    """(relative error of Y, microseconds of a step)."""
    b = Block(d, f, n_experts, top_k, tokens)
    b.X.normal_()
    b.forward()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.forward()
    b.Y.zero_()
    graph.replay()
    torch.cuda.synchronize()
    y = b.exact()
    err = float((b.Y.double() - y).norm() / y.norm())
    t = time.perf_counter()
    for _ in range(steps):
        graph.replay()
    torch.cuda.synchronize()
    return err, (time.perf_counter() - t) / steps * 1e6


if __name__ == "__main__":
    for n in (1, 8, 64):
        e, us = run(2048, 768, 64, 6, n)
        print(f"{n:3d} tokens: relative error {e:.2e}, {us:.1f} us a step", flush=True)
