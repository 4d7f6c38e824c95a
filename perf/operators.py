"""Cases of the FP8 operators: the block-scaled linear layer and the mixture-of-experts layer.

linear   Y = Q(X) Q(W)^T with E4M3 codes, one activation scale per token and 128 inputs, one
         weight scale per 128 x 128 block.  Weights are given as codes and scales (a
         quantized checkpoint); the activations are quantized within the call.
moe      router logits, top-k experts of each token, the experts' up projections (gated
         SiLU, or GELU-tanh), their down projections, and the weighted sum, for a few tokens.
         Weights are E4M3 codes with one scale per 128 x 128 block; activations stay bf16.

`own` false computes both from elementary torch operations in 32 bits; `own` true calls the
library.  Scale kinds: "f32" (amax / 448) and "e8m0" (the smallest power of two that keeps
the block within 448).
"""
import math

import torch

own = False

E4M3_MAX = 448.0
TINY = 2.0 ** -60           # smallest scale: products of two scales stay normal binary32 numbers
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _linear(name, T, d_in, d_out, x, y, scales):
    return {"name": name, "op": "linear", "T": T, "d_in": d_in, "d_out": d_out, "x": x, "y": y, "scales": scales}


def _moe(name, T, d, f, E, k, act, x, renorm):
    return {"name": name, "op": "moe", "T": T, "d": d, "f": f, "E": E, "k": k, "act": act, "x": x, "renorm": renorm}


def listed():
    return [
        # one token through the FFN up projection: the weights' bytes are all that counts
        _linear("linear one token", 1, 5120, 13824, "bf16", "bf16", "f32"),
        # a small batch of tokens through the down projection, fp32 out for a residual sum
        _linear("linear 24 tokens", 24, 13824, 5120, "bf16", "f32", "f32"),
        # the tiny workload's layer: a call that is all latency
        _linear("linear tiny layer", 256, 512, 1024, "f32", "f32", "f32"),
        # odd sizes: rows that are not 16-byte aligned, blocks cut by both edges
        _linear("linear odd sizes", 333, 4999, 1111, "bf16", "bf16", "f32"),
        # a 4096-token pass, down projection, power-of-two scales
        _linear("linear 4096 tokens, down, e8m0", 4096, 13824, 5120, "bf16", "bf16", "e8m0"),
        # a 4096-token pass, up projection, fp32 out
        _linear("linear 4096 tokens, up", 4096, 5120, 13824, "bf16", "f32", "f32"),
        # the full token count of a video frame stack
        _linear("linear 57600 tokens, up", 57600, 5120, 13824, "bf16", "bf16", "f32"),
        # one token through a layer of many experts: eight of 64 are read
        _moe("moe one token", 1, 5120, 1536, 64, 8, "silu", "bf16", True),
        # a few tokens, small experts, router probabilities over all experts
        _moe("moe 8 tokens, small experts", 8, 2048, 768, 128, 8, "silu", "bf16", False),
        # a few tokens through few wide experts with the FFN block's GELU-tanh
        _moe("moe 16 tokens, wide experts", 16, 5120, 13824, 8, 2, "gelu", "bf16", True),
        # odd sizes, fp32 activations
        _moe("moe odd sizes", 37, 1000, 333, 10, 3, "silu", "f32", True),
        # a decoding batch: nearly every expert is read
        _moe("moe 64 tokens", 64, 5120, 1536, 64, 6, "silu", "bf16", True),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    while True:
        if rng.random() < 0.55:
            c = _linear("", _log(rng, 1, 57600), _log(rng, 128, 13824), _log(rng, 16, 13824), rng.choice(["bf16", "bf16", "f32"]),
                        rng.choice(["bf16", "f32"]), rng.choice(["f32", "f32", "e8m0"]))
            # at most the largest listed product
            if c["T"] * c["d_in"] * c["d_out"] > 57600 * 5120 * 13824:
                continue
        else:
            E = _log(rng, 4, 128)
            c = _moe("", _log(rng, 1, 64), _log(rng, 256, 5120), _log(rng, 64, 13824), E, rng.randint(1, min(8, E)),
                     rng.choice(["silu", "silu", "gelu"]), rng.choice(["bf16", "bf16", "f32"]), rng.random() < 0.6)
            # at most the largest listed layer's weights
            if c["E"] * c["d"] * c["f"] > 64 * 5120 * 1536:
                continue
        del c["name"]
        return c


# --------------------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _pow2_code(amax):
    """E8M0 code of the smallest power of two s with amax <= 448 s, s >= 2^-60."""
    m, e = torch.frexp(amax)                 # amax = 2m * 2^(e-1), 448 = 1.75 * 2^8
    c = e - 9 + (m > 0.875).to(torch.int32) + 127
    return torch.clamp(c, 127 - 60, 254).to(torch.uint8)


def _quantized(n, rows, cols, std, scales, g):
    """n random [rows, cols] matrices as E4M3 codes and their 128 x 128 block scales."""
    rb, cb = -(-rows // 128), -(-cols // 128)
    codes = torch.empty(n, rows, cols, dtype=torch.uint8, device="cuda")
    sc = torch.empty(n, rb, cb, dtype=torch.float32 if scales == "f32" else torch.uint8, device="cuda")
    for i in range(n):
        w = torch.zeros(rb * 128, cb * 128, device="cuda")
        w[:rows, :cols] = torch.randn(rows, cols, device="cuda", generator=g) * std
        blocks = w.view(rb, 128, cb, 128)
        amax = blocks.abs().amax(dim=(1, 3))
        if scales == "f32":
            sc[i] = amax / E4M3_MAX
            s = sc[i]
        else:
            sc[i] = _pow2_code(amax)
            s = (sc[i].to(torch.int32) << 23).view(torch.float32)
        q = (blocks / s[:, None, :, None]).view(rb * 128, cb * 128)[:rows, :cols]
        codes[i] = q.to(torch.float8_e4m3fn).view(torch.uint8)
    return codes, sc


def _acts(T, d, dtype, g):
    """Tokens with a few heavy channels, as the inputs of a transformer's projections have."""
    x = torch.randn(T, d, device="cuda", generator=g) * 0.3
    heavy = torch.randperm(d, device="cuda", generator=g)[:max(1, d // 80)]
    x[:, heavy] *= 12.0
    return x.clamp_(-12.0, 12.0).to(dtype)


def prepare(case, seed):
    g = _gen(seed)
    if case["op"] == "linear":
        T, d_in, d_out = case["T"], case["d_in"], case["d_out"]
        st = {"case": case, "X": _acts(T, d_in, DTYPES[case["x"]], g)}
        codes, sc = _quantized(1, d_out, d_in, 0.02, case["scales"], g)
        st["codes"], st["sc"] = codes[0], sc[0]
        if own:
            from bit_quantized_dit_amd import w4a4 as B
            st["layer"] = B.w4a4_fp8_pack_codes(st["codes"], st["sc"])
            st["ws"] = B.alloc_workspace_fp8(T, st["layer"])
            st["Y"] = torch.empty(T, d_out, dtype=DTYPES[case["y"]], device="cuda")
        return st
    T, d, f, E = case["T"], case["d"], case["f"], case["E"]
    st = {"case": case, "X": _acts(T, d, DTYPES[case["x"]], g)}
    # logits of a spread that leaves the chosen experts with unequal weights
    st["router"] = (torch.randn(E, d, device="cuda", generator=g) * (2.0 / math.sqrt(d))).to(torch.bfloat16)
    if case["act"] == "silu":
        st["gate"] = _quantized(E, f, d, 0.02, "f32", g)
    st["up"] = _quantized(E, f, d, 0.02, "f32", g)
    st["down"] = _quantized(E, d, f, 0.02, "f32", g)
    if own:
        from bit_quantized_dit_amd import w4a4 as B
        st["layer"] = B.moe_layer(st["router"], B.w4a4_fp8_pack_codes(*st["gate"]) if "gate" in st else None,
                                  B.w4a4_fp8_pack_codes(*st["up"]), B.w4a4_fp8_pack_codes(*st["down"]),
                                  top_k=case["k"], renormalize=case["renorm"])
        st["ws"] = B.alloc_workspace_moe(T, st["layer"])
        st["Y"] = torch.empty(T, d, dtype=torch.bfloat16, device="cuda")
    return st


# --------------------------------------------------------------------------- plain form

def _dequant(codes, sc):
    """fp32 values of E4M3 codes [..., rows, cols] with 128 x 128 block scales."""
    s = sc if sc.dtype == torch.float32 else (sc.to(torch.int32) << 23).view(torch.float32)
    rows, cols = codes.shape[-2:]
    w = codes.view(torch.float8_e4m3fn).to(torch.float32)
    w *= s.repeat_interleave(128, -2)[..., :rows, :].repeat_interleave(128, -1)[..., :cols]
    return w


def _plain_linear(st):
    case, X = st["case"], st["X"]
    T, d_in = X.shape
    kb = -(-d_in // 128)
    x = torch.nn.functional.pad(X.to(torch.float32), (0, kb * 128 - d_in)).view(T, kb, 128)
    amax = x.abs().amax(dim=2, keepdim=True)
    if case["scales"] == "f32":
        s = (amax / torch.full_like(amax, E4M3_MAX)).clamp_min(TINY)      # a true division: one by a number is a product
    else:
        s = (_pow2_code(amax).to(torch.int32) << 23).view(torch.float32)
    xq = ((x / s).to(torch.float8_e4m3fn).to(torch.float32) * s).view(T, kb * 128)[:, :d_in]
    return (xq @ _dequant(st["codes"], st["sc"]).t()).to(DTYPES[case["y"]])


def _activation(g, u):
    if g is not None:
        return g / (1.0 + torch.exp(-g)) * u
    return 0.5 * u * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (u + 0.044715 * u * u * u)))


def _route(case, logits):
    val, ids = torch.sort(logits, dim=1, descending=True, stable=True)
    p = torch.exp(logits - val[:, :1])
    sel = torch.gather(p, 1, ids[:, :case["k"]])
    return ids[:, :case["k"]], sel / (sel if case["renorm"] else p).sum(dim=1, keepdim=True)


def _plain_moe(st):
    case, X = st["case"], st["X"]
    T, d, f, E, k = case["T"], case["d"], case["f"], case["E"], case["k"]
    ids, p = _route(case, X.to(torch.float32) @ st["router"].to(torch.float32).t())
    xb = X.to(torch.bfloat16).to(torch.float32)
    if T * k <= E:      # few pairs: the chosen experts' weights, pair by pair
        at = ids.reshape(-1)
        xs = xb.repeat_interleave(k, 0).unsqueeze(2)
        prod = lambda w, v: torch.bmm(_dequant(w[0][at], w[1][at]), v)
        h = _activation(prod(st["gate"], xs) if "gate" in st else None, prod(st["up"], xs))
        y = prod(st["down"], h.to(torch.bfloat16).to(torch.float32)).view(T, k, d)
        return (y * p.unsqueeze(2)).sum(dim=1).to(torch.bfloat16)
    # many pairs: every expert on every token, the others' weights zero
    prod = lambda w: xb @ _dequant(*w).view(E * f, d).t()
    h = _activation(prod(st["gate"]) if "gate" in st else None, prod(st["up"])).to(torch.bfloat16).to(torch.float32)
    pe = torch.zeros(T, E, device="cuda").scatter_(1, ids, p)
    h = (h.view(T, E, f) * pe.unsqueeze(2)).view(T, E * f)
    return (h @ _dequant(*st["down"]).transpose(1, 2).reshape(E * f, d)).to(torch.bfloat16)


def run(state):
    if not own:
        return _plain_linear(state) if state["case"]["op"] == "linear" else _plain_moe(state)
    from bit_quantized_dit_amd import w4a4 as B
    call = B.w4a4_fp8_linear if state["case"]["op"] == "linear" else B.w4a4_moe_forward
    call(state["X"], state["layer"], state["Y"], state["ws"])
    return state["Y"]


def work(case):
    size = {"bf16": 2, "f32": 4}
    if case["op"] == "linear":
        T, d_in, d_out = case["T"], case["d_in"], case["d_out"]
        blocks = -(-d_in // 128) * -(-d_out // 128)
        return {"bytes": T * d_in * size[case["x"]] + d_in * d_out + blocks * (4 if case["scales"] == "f32" else 1) + T * d_out * size[case["y"]],
                "flops": 2 * T * d_in * d_out}
    T, d, f, E, k = case["T"], case["d"], case["f"], case["E"], case["k"]
    mats = 3 if case["act"] == "silu" else 2
    read = E * (1.0 - (1.0 - k / E) ** T)      # experts that at least one token chose, on average
    return {"bytes": read * mats * d * f + 2 * E * d + T * d * (size[case["x"]] + 2), "flops": 2 * T * k * mats * d * f + 2 * T * E * d}


# --------------------------------------------------------------------------- 64 bits

def _value64(codes):
    """E4M3 codes as float64, from their bit fields."""
    c = codes.to(torch.int64)
    e, m = (c >> 3) & 15, (c & 7).double()
    v = torch.where(e == 0, m * 2.0 ** -9, (1.0 + m / 8.0) * torch.exp2((e - 7).double()))
    return torch.where(c >= 128, -v, v)


def _scale64(sc):
    return sc.double() if sc.dtype == torch.float32 else torch.exp2(sc.double() - 127.0)


def _weights64(codes, sc):
    w = _value64(codes)
    rows, cols = w.shape
    i, j = torch.arange(rows, device=w.device) // 128, torch.arange(cols, device=w.device) // 128
    return w * _scale64(sc)[i][:, j]


def _nearest64(q):
    """The E4M3 value nearest to q, ties to the even mantissa, |q| at most 448 and a rounding."""
    e = torch.floor(torch.log2(q.abs().clamp_min(2.0 ** -6)))
    e = torch.where(q.abs() >= torch.exp2(e + 1), e + 1, torch.where(q.abs() < torch.exp2(e), e - 1, e)).clamp_min(-6.0)
    step = torch.exp2(e - 3)
    return (torch.round(q / step) * step).clamp(-448.0, 448.0)


def _linear64(st):
    case, X = st["case"], st["X"]
    w = _weights64(st["codes"], st["sc"])
    out = torch.empty(case["T"], case["d_out"], dtype=torch.float64, device="cuda")
    for t0 in range(0, case["T"], 8192):
        x = X[t0:t0 + 8192].double()
        for j in range(0, case["d_in"], 128):
            b = x[:, j:j + 128]
            amax = b.abs().amax(dim=1, keepdim=True)
            if case["scales"] == "f32":     # binary32: amax / 448 rounded once
                s = (amax / 448.0).float().double().clamp_min(2.0 ** -60)
            else:
                s = torch.exp2(torch.ceil(torch.log2((amax / 448.0).clamp_min(2.0 ** -60))))
                s = torch.where(amax > 448.0 * s, 2 * s, torch.where((amax <= 224.0 * s) & (s > 2.0 ** -60), s / 2, s))
            x[:, j:j + 128] = _nearest64((b / s).float().double()) * s
        out[t0:t0 + 8192] = x @ w.t()
    return out


def _moe64(st):
    case, X = st["case"], st["X"]
    x = X.double()
    logits = x @ st["router"].double().t()
    order = torch.argsort(logits, dim=1, descending=True, stable=True)
    chosen = torch.zeros_like(logits).scatter_(1, order[:, :case["k"]], 1.0)
    p = torch.softmax(logits, dim=1) * chosen
    if case["renorm"]:
        p = p / p.sum(dim=1, keepdim=True)
    xb = X.to(torch.bfloat16).double()
    y = torch.zeros(case["T"], case["d"], dtype=torch.float64, device="cuda")
    for e in range(case["E"]):
        t = torch.nonzero(chosen[:, e]).flatten()
        if not len(t):
            continue
        u = xb[t] @ _weights64(st["up"][0][e], st["up"][1][e]).t()
        if "gate" in st:
            g = xb[t] @ _weights64(st["gate"][0][e], st["gate"][1][e]).t()
            h = g * torch.sigmoid(g) * u
        else:
            h = torch.nn.functional.gelu(u, approximate="tanh")
        y[t] += p[t, e, None] * (h.to(torch.bfloat16).double() @ _weights64(st["down"][0][e], st["down"][1][e]).t())
    return y


def exact(case, seed):
    global own
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    return _linear64(st) if case["op"] == "linear" else _moe64(st)
