"""The attention of a transformer block with its operators together, as a user runs them: one quantization
for the query, key and value projections (INT8), rows appended to the 4-bit cache, attention over it,
the output projection; a prompt first, then tokens one by one from a HIP graph.  Every step is compared
with 64-bit forms that start from what the step before left."""
import numpy as np
import pytest
import torch

from bit_quantized_dit_amd import w4a4 as B
from tests import kv_ref as R

pytestmark = pytest.mark.gpu


def _linear64(x, layer):
    q, s = R.int8_quantize(x.float().cpu().numpy())
    v = layer.views()
    return R.int8_product(q, s, v["codes"].cpu().numpy(), v["scales"].cpu().numpy())


class Block:
    """d -> (Hq + 2 H) D, attention, Hq D -> d."""

    def __init__(self, d, Hq, H, D, seqs, tokens, page=16):
        g = torch.Generator(device="cuda").manual_seed(4)
        self.d, self.Hq, self.H, self.D = d, Hq, H, D
        w = lambda n, k: torch.randn(n, k, device="cuda", generator=g) * k ** -0.5
        self.qkv, self.out = B.w4a4_int8_pack_weights(w((Hq + 2 * H) * D, d)), B.w4a4_int8_pack_weights(w(d, Hq * D))
        per = -(-tokens // page)
        self.cache = B.kv_cache(seqs * per, page, H, D)
        self.pages = torch.randperm(seqs * per, device="cuda", generator=g).to(torch.int32).view(seqs, per)
        self.lens = torch.zeros(seqs, dtype=torch.int32, device="cuda")
        self.kept = [[np.zeros((0, H, D), np.float32)] * 2 for _ in range(seqs)]

    def plan(self, rows, max_rows):
        n = sum(rows)
        start = torch.tensor(np.cumsum([0] + rows), dtype=torch.int32, device="cuda")
        p = {"rows": rows, "X": torch.zeros(n, self.d, dtype=torch.bfloat16, device="cuda"), "batch": B.kv_batch(start, self.lens, self.pages, max_rows)}
        p["F"] = torch.empty(n, (self.Hq + 2 * self.H) * self.D, dtype=torch.bfloat16, device="cuda")
        p["O"] = torch.empty(n, self.Hq, self.D, dtype=torch.bfloat16, device="cuda")
        p["Y"] = torch.empty(n, self.d, device="cuda")
        p["ws"] = [B.alloc_workspace_int8(n, self.qkv), B.alloc_workspace_kv(n, p["batch"], self.Hq, self.cache), B.alloc_workspace_int8(n, self.out)]
        return p

    def run(self, p):
        n = sum(p["rows"])
        B.w4a4_int8_linear(p["X"], self.qkv, p["F"], p["ws"][0])
        heads = p["F"].view(n, self.Hq + 2 * self.H, self.D)
        B.w4a4_kv_append(heads[:, self.Hq:self.Hq + self.H], heads[:, self.Hq + self.H:], p["batch"], self.cache)
        B.w4a4_kv_attention(heads[:, :self.Hq], p["batch"], self.cache, p["O"], p["ws"][1])
        B.w4a4_int8_linear(p["O"].view(n, -1), self.out, p["Y"], p["ws"][2])

    def check(self, p):
        torch.cuda.synchronize()
        n, Hq, H, D = sum(p["rows"]), self.Hq, self.H, self.D
        y, tol = _linear64(p["X"], self.qkv)
        F = p["F"].double().cpu().numpy()
        assert (np.abs(F - y) <= tol + R.BF16_U * (np.abs(y) + tol)).all()
        heads = F.reshape(n, -1, D).astype(np.float32)
        few = p["batch"].desc.max_rows * (Hq // H) <= 64
        at = 0
        for i, r in enumerate(p["rows"]):
            self.kept[i] = [np.concatenate([old, heads[at:at + r, a:a + H]]) for old, a in zip(self.kept[i], (Hq, Hq + H))]
            k, v = (R.mxfp4(x)[2] for x in self.kept[i])
            L = len(k)
            assert L == int(self.lens[i])
            for h in range(Hq):
                o, t, _ = R.attention(heads[at:at + r, h], k[:, h // (Hq // H)], v[:, h // (Hq // H)], D ** -0.5, np.zeros(r, int), np.arange(L - r, L) + 1, few)
                assert bool(((p["O"][at:at + r, h].double().cpu() - o).abs() <= t).all()), (i, h)
            at += r
        y, tol = _linear64(p["O"].view(n, -1), self.out)
        assert (np.abs(p["Y"].double().cpu().numpy() - y) <= tol).all()


@pytest.mark.parametrize("d,Hq,H,D,prompts", [(640, 5, 5, 128, [70, 3, 130]), (520, 8, 2, 72, [33, 200])])
def test_prompt_then_tokens(d, Hq, H, D, prompts):
    blk = Block(d, Hq, H, D, len(prompts), max(prompts) + 8)
    p = blk.plan(prompts, max(prompts))
    p["X"].normal_()
    blk.lens += torch.tensor(prompts, dtype=torch.int32, device="cuda")
    blk.run(p)
    blk.check(p)
    p = blk.plan([1] * len(prompts), 1)
    p["X"].normal_()
    blk.lens += 1
    blk.run(p)
    blk.check(p)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        blk.run(p)
    for _ in range(4):
        p["X"].normal_()
        blk.lens += 1
        graph.replay()
        blk.check(p)
