"""Cases of the attention block's quantized operators: the INT8 linear layer, the 4-bit key/value
cache and attention over it.

int8    Y = Q(X) Q(W)^T with 8-bit integer codes, one scale per token and one per output
        channel.  Weights are given as codes and scales (a quantized checkpoint); the
        activations are quantized within the call.
cache   rows of keys and values quantized to MXFP4 (E2M1 codes, an E8M0 scale per 32 channels
        of a head) as they are written into a paged cache, and the same rows read back.
read    whole sequences read back out of the cache.
attn    attention of each sequence's last rows over its cached keys and values: one row
        (decoding), or many (a prompt, or a chunk of one), causal, windowed or neither.

Row i of a sequence with n rows and `len` cached tokens stands at position len - n + i.

`own` false computes them from elementary torch operations in 32 bits; `own` true calls the
library.
"""
import math
import random

import torch

own = False

TINY = 2.0 ** -60           # smallest scale of the 8-bit codes
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _int8(name, T, d_in, d_out, x, y):
    return {"name": name, "op": "int8", "T": T, "d_in": d_in, "d_out": d_out, "x": x, "y": y}


def _store(name, op, seqs, rows, lens, kv_heads, d, page, x, y):
    """rows and lens: (smallest, largest) of a sequence; the others are spread evenly between."""
    return {"name": name, "op": op, "seqs": seqs, "rows_lo": rows[0], "rows_hi": rows[1], "len_lo": lens[0], "len_hi": lens[1],
            "kv_heads": kv_heads, "d": d, "page": page, "x": x, "y": y}


def _attn(name, seqs, rows, lens, heads, kv_heads, d, page, causal, window, q):
    return {"name": name, "op": "attn", "seqs": seqs, "rows_lo": rows[0], "rows_hi": rows[1], "len_lo": lens[0], "len_hi": lens[1],
            "heads": heads, "kv_heads": kv_heads, "d": d, "page": page, "causal": causal, "window": window, "q": q}


def listed():
    return [
        # one token through a projection: the weights' bytes are all that counts
        _int8("int8 one token", 1, 5120, 13824, "bf16", "bf16"),
        # odd sizes: rows that are not 16-byte aligned, tiles cut by both edges, fp32 in and out
        _int8("int8 odd sizes", 333, 4999, 1111, "f32", "f32"),
        # the output projection at the full token count of a video frame stack
        _int8("int8 57600 tokens", 57600, 5120, 5120, "bf16", "bf16"),
        # a decoding batch's new rows: a call that is all latency
        _store("cache decoding rows", "cache", 64, (1, 1), (100, 4000), 8, 128, 16, "bf16", "bf16"),
        # a frame stack's keys and values
        _store("cache prompt", "cache", 1, (57600, 57600), (57600, 57600), 40, 128, 256, "bf16", "bf16"),
        # a few sequences back out, a head width that its scale groups do not divide, fp32
        _store("read odd heads", "read", 7, (100, 9000), (100, 9000), 6, 72, 48, "bf16", "f32"),
        # one long sequence back out
        _store("read long", "read", 1, (57600, 57600), (57600, 57600), 40, 128, 256, "bf16", "bf16"),
        # one row of a short sequence: latency
        _attn("attn one short row", 1, (1, 1), (500, 500), 32, 8, 128, 16, True, 0, "bf16"),
        # one row over the whole frame stack, a key/value head for each head
        _attn("attn one long row", 1, (1, 1), (57600, 57600), 40, 40, 128, 256, True, 0, "bf16"),
        # a decoding batch of ragged sequences, five query heads to a key/value head
        _attn("attn decoding batch", 64, (1, 1), (512, 32768), 40, 8, 128, 64, True, 0, "bf16"),
        # ragged prompts, odd head width, a window, fp32 queries
        _attn("attn odd prompts", 5, (1, 777), (200, 2100), 12, 4, 72, 48, True, 256, "f32"),
        # a chunk of rows that sees the whole frame stack, as a video block does
        _attn("attn chunk", 1, (4096, 4096), (57600, 57600), 40, 40, 128, 256, False, 0, "bf16"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _pair(rng, lo, hi):
    a, b = _log(rng, lo, hi), _log(rng, lo, hi)
    return min(a, b), max(a, b)


def draw(rng):
    while True:
        kind = rng.choice(["int8", "cache", "read", "attn", "attn", "attn"])
        if kind == "int8":
            c = _int8("", _log(rng, 1, 57600), _log(rng, 128, 13824), _log(rng, 16, 13824), rng.choice(["bf16", "bf16", "f32"]),
                      rng.choice(["bf16", "f32"]))
            if c["T"] * c["d_in"] * c["d_out"] > 57600 * 5120 * 5120:
                continue
        else:
            seqs, H = _log(rng, 1, 64), _log(rng, 1, 40)
            d, page = rng.choice([64, 72, 80, 96, 128, 128, 128, 256]), rng.choice([16, 48, 64, 128, 256])
            lens = _pair(rng, 16, 57600)
            decode = kind != "attn" or rng.random() < 0.5
            rows = lens if kind == "read" else (1, rng.choice([1, 1, 1, 2, 4])) if decode and kind == "attn" else _pair(rng, 1, 4096)
            if kind == "attn":
                c = _attn("", seqs, rows, lens, H * rng.choice([1, 1, 2, 4, 5, 8]), H, d, page, rng.random() < 0.7,
                          rng.choice([0, 0, 256, 1000]), rng.choice(["bf16", "bf16", "f32"]))
                if not c["causal"]:
                    c["window"] = 0
                # at most the longest listed cache and a quarter of the largest listed product
                if c["heads"] > 64 or seqs * lens[1] * H * d > 64 * 16640 * 8 * 128 or work(c)["flops"] > 1.2e12:
                    continue
                # the plain form takes sequences one by one: few of them where there are many rows
                if not decode and seqs > 16:
                    continue
            else:
                c = _store("", kind, seqs, rows, lens, H, d, page, rng.choice(["bf16", "f32"]), rng.choice(["bf16", "f32"]))
                if seqs * max(lens[1], rows[1]) * H * d > 57600 * 40 * 128:
                    continue
        del c["name"]
        return c


# --------------------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _spread(lo, hi, n):
    return [lo + (hi - lo) * i // max(1, n - 1) for i in range(n)]


def _sizes(case):
    """(rows, lens) of the sequences, smallest first."""
    lens = _spread(case["len_lo"], case["len_hi"], case["seqs"])
    if case["op"] == "read":
        return lens, lens
    rows = _spread(case["rows_lo"], case["rows_hi"], case["seqs"])
    if case["op"] == "cache":
        return rows, [max(n, r) for n, r in zip(lens, rows)]
    return [min(n, r) for n, r in zip(lens, rows)], lens


def _batch(case, seed):
    """The sequences in an order of the seed's, and pages of a pool in an order of its own."""
    rng = random.Random(seed)
    pairs = list(zip(*_sizes(case)))
    rng.shuffle(pairs)
    page = case["page"]
    need = [-(-n // page) for _, n in pairs]
    n_pages = sum(need) + 3
    perm = torch.randperm(n_pages, generator=torch.Generator().manual_seed(seed)).to(torch.int32)
    table = torch.zeros(len(pairs), max(need), dtype=torch.int32)
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = perm[at:at + n]
        at += n
    start = [0]
    for r, _ in pairs:
        start.append(start[-1] + r)
    return {"rows": [r for r, _ in pairs], "lens": [n for _, n in pairs], "n_pages": n_pages, "T": start[-1],
            "q_start": torch.tensor(start, dtype=torch.int32, device="cuda"),
            "lens_dev": torch.tensor([n for _, n in pairs], dtype=torch.int32, device="cuda"), "table": table.cuda()}


def _heads(T, H, d, g, heavy, std=1.0):
    """Rows of H heads; keys have a few heavy channels."""
    x = torch.randn(T, H, d, device="cuda", generator=g) * std
    if heavy:
        x[:, :, torch.randperm(d, device="cuda", generator=g)[:max(1, d // 32)]] *= 3.0
    return x


def _acts(T, d, dtype, g):
    """Tokens with a few heavy channels, as the inputs of a transformer's projections have."""
    x = torch.randn(T, d, device="cuda", generator=g) * 0.3
    heavy = torch.randperm(d, device="cuda", generator=g)[:max(1, d // 80)]
    x[:, heavy] *= 12.0
    return x.clamp_(-12.0, 12.0).to(dtype)


def _int8_inputs(case, seed):
    g = _gen(seed)
    X = _acts(case["T"], case["d_in"], DTYPES[case["x"]], g)
    W = torch.randn(case["d_out"], case["d_in"], device="cuda", generator=g) * 0.02
    s = W.abs().amax(dim=1) / 127.0
    return X, (W / s[:, None]).round_().clamp_(-127, 127).to(torch.int8), s


def _kv_inputs(case, seed):
    """The batch, and keys and values of every token that has to be in the cache: of all sequences'
    tokens, or of the new rows where the call itself writes them."""
    b, g = _batch(case, seed), _gen(seed)
    n = b["T"] if case["op"] == "cache" else sum(b["lens"])
    dt = DTYPES[case["x"]] if "x" in case else torch.bfloat16
    K = _heads(n, case["kv_heads"], case["d"], g, True).to(dt)
    V = _heads(n, case["kv_heads"], case["d"], g, False).to(dt)
    Q = _heads(b["T"], case["heads"], case["d"], g, False, 1.5).to(DTYPES[case["q"]]) if case["op"] == "attn" else None
    return b, K, V, Q


def prepare(case, seed):
    if case["op"] == "int8":
        X, codes, s = _int8_inputs(case, seed)
        st = {"case": case, "X": X, "codes": codes, "s": s}
        if own:
            from bit_quantized_dit_amd import w4a4 as B
            st["layer"] = B.w4a4_int8_pack_codes(codes, s)
            st["ws"] = B.alloc_workspace_int8(case["T"], st["layer"])
            st["Y"] = torch.empty(case["T"], case["d_out"], dtype=DTYPES[case["y"]], device="cuda")
        return st
    b, K, V, Q = _kv_inputs(case, seed)
    T, H, d = b["T"], case["kv_heads"], case["d"]
    st = {"case": case, "b": b, "Q": Q}
    if case["op"] == "cache":
        st["K"], st["V"] = K, V
    fill_start = torch.tensor([0] + b["lens"], device="cuda").cumsum(0).to(torch.int32)      # every sequence from its first token
    if own:
        from bit_quantized_dit_amd import w4a4 as B
        st["cache"] = B.kv_cache(b["n_pages"], case["page"], H, d)
        st["batch"] = B.kv_batch(b["q_start"], b["lens_dev"], b["table"], max_rows=max(b["rows"]))
        if case["op"] != "cache":
            B.w4a4_kv_append(K, V, B.kv_batch(fill_start, b["lens_dev"], b["table"], max_rows=max(b["lens"])), st["cache"])
        if case["op"] == "attn":
            st["ws"] = B.alloc_workspace_kv(T, st["batch"], case["heads"], st["cache"])
            st["O"] = torch.empty(T, case["heads"], d, dtype=torch.bfloat16, device="cuda")
        else:
            st["Kout"], st["Vout"] = (torch.empty(T, H, d, dtype=DTYPES[case["y"]], device="cuda") for _ in range(2))
        return st
    G = -(-d // 32)
    slots = b["n_pages"] * case["page"]
    st["cache"] = {n: (torch.zeros(slots, H, 16 * G, dtype=torch.uint8, device="cuda"),
                       torch.zeros(slots, H, G, dtype=torch.uint8, device="cuda")) for n in ("K", "V")}
    if case["op"] != "cache":
        at = _slots(fill_start, b["lens_dev"], b["table"], case["page"], len(K))
        _plain_append(st["cache"]["K"], at, K)
        _plain_append(st["cache"]["V"], at, V)
    return st


# --------------------------------------------------------------------------- plain form

def _plain_int8(st):
    x = st["X"].to(torch.float32)
    amax = x.abs().amax(dim=1, keepdim=True)
    s = (amax / torch.full_like(amax, 127.0)).clamp_min(TINY)      # a true division: one by a number is a product
    q = torch.round(x / s)
    return ((q @ st["codes"].to(torch.float32).t()) * (s * st["s"])).to(DTYPES[st["case"]["y"]])


def _slots(q_start, lens, table, page, T):
    """Where in the cache each of the T rows stands."""
    rows = torch.arange(T, device=q_start.device)
    b = torch.searchsorted(q_start[1:].long(), rows, right=True)
    pos = lens.long()[b] - q_start[b + 1].long() + rows
    return table[b, pos // page].long() * page + pos % page


_BLOCK = 1 << 13            # rows at a time, so that the 32-bit steps stay small beside the cache


def _plain_append(cache, at, X):
    codes, scales = cache
    H, G = scales.shape[1:]
    for t0 in range(0, len(X), _BLOCK):
        x = X[t0:t0 + _BLOCK].to(torch.float32)
        x = torch.nn.functional.pad(x, (0, 32 * G - x.shape[2])).view(len(x), H, G, 32)
        a = x.abs()
        c = torch.clamp((a.amax(dim=3).view(torch.int32) >> 23) - 2, min=0)      # floor(log2 amax) - 2, biased
        y = a * torch.exp2(127.0 - c.to(torch.float32)).unsqueeze(3)
        m = (y > 0.25).to(torch.uint8)
        for up, tie in ((0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True), (5.0, False)):
            m += (y >= up) if tie else (y > up)
        m += (x < 0).to(torch.uint8) * 8
        m = m.view(len(x), H, 16 * G, 2)
        codes[at[t0:t0 + _BLOCK]] = m[..., 0] | (m[..., 1] << 4)
        scales[at[t0:t0 + _BLOCK]] = c.to(torch.uint8)


def _plain_read(cache, at, d):
    """fp32 values [rows, H, d] of the slots."""
    codes, scales = cache
    m = codes[at]
    H, G = scales.shape[1:]
    value = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device=m.device)
    value = torch.cat([value, -value])
    v = value[torch.stack([m & 15, m >> 4], dim=3).int()].view(len(at), H, G, 32)
    return (v * torch.exp2(scales[at].to(torch.float32) - 127.0).unsqueeze(3)).view(len(at), H, 32 * G)[..., :d]


def _plain_store(st):
    case, b = st["case"], st["b"]
    at = _slots(b["q_start"], b["lens_dev"], b["table"], case["page"], b["T"])
    out = []
    for n in ("K", "V"):
        if case["op"] == "cache":
            _plain_append(st["cache"][n], at, st[n])
        o = torch.empty(b["T"], case["kv_heads"], case["d"], dtype=DTYPES[case["y"]], device="cuda")
        for t0 in range(0, b["T"], _BLOCK):
            o[t0:t0 + _BLOCK] = _plain_read(st["cache"][n], at[t0:t0 + _BLOCK], case["d"])
        out.append(o)
    return out


def _plain_attn(st):
    case, b = st["case"], st["b"]
    H, d, page = case["kv_heads"], case["d"], case["page"]
    G = case["heads"] // H
    out, t = [], 0
    for i, (n, L) in enumerate(zip(b["rows"], b["lens"])):
        pos = torch.arange(L, device="cuda")
        at = b["table"][i, pos // page].long() * page + pos % page
        k = _plain_read(st["cache"]["K"], at, d).permute(1, 2, 0)          # [H, d, L]
        v = _plain_read(st["cache"]["V"], at, d).permute(1, 0, 2)          # [H, L, d]
        q = st["Q"][t:t + n].to(torch.bfloat16).to(torch.float32).view(n, H, G, d).permute(1, 2, 0, 3).reshape(H, G * n, d)
        here = (L - n + torch.arange(n, device="cuda")).repeat(G)
        seen = None
        if case["causal"]:
            seen = pos[None] <= here[:, None]
            if case["window"]:
                seen &= pos[None] > here[:, None] - case["window"]
        o = torch.empty(H, G * n, d, device="cuda")
        step = max(1, (1 << 29) // (G * n * L))
        for h in range(0, H, step):
            s = torch.bmm(q[h:h + step], k[h:h + step].contiguous()) * (1.0 / math.sqrt(d))
            if seen is not None:
                s = torch.where(seen, s, torch.full_like(s, -math.inf))
            p = torch.exp(s - s.amax(dim=2, keepdim=True))
            o[h:h + step] = torch.bmm(p, v[h:h + step].contiguous()) / p.sum(dim=2, keepdim=True)
        out.append(o.view(H, G, n, d).permute(2, 0, 1, 3).reshape(n, H * G, d).to(torch.bfloat16))
        t += n
    return torch.cat(out)


def run(state):
    op = state["case"]["op"]
    if not own:
        return _plain_int8(state) if op == "int8" else _plain_attn(state) if op == "attn" else _plain_store(state)
    from bit_quantized_dit_amd import w4a4 as B
    if op == "int8":
        B.w4a4_int8_linear(state["X"], state["layer"], state["Y"], state["ws"])
        return state["Y"]
    if op == "attn":
        c = state["case"]
        B.w4a4_kv_attention(state["Q"], state["batch"], state["cache"], state["O"], state["ws"], causal=c["causal"], window=c["window"])
        return state["O"]
    if op == "cache":
        B.w4a4_kv_append(state["K"], state["V"], state["batch"], state["cache"])
    B.w4a4_kv_read(state["batch"], state["cache"], state["Kout"], state["Vout"])
    return [state["Kout"], state["Vout"]]


def work(case):
    size = {"bf16": 2, "f32": 4}
    if case["op"] == "int8":
        T, d_in, d_out = case["T"], case["d_in"], case["d_out"]
        return {"bytes": T * d_in * size[case["x"]] + d_in * d_out + 4 * d_out + T * d_out * size[case["y"]], "flops": 2 * T * d_in * d_out}
    rows, lens = _sizes(case)
    H, d = case["kv_heads"], case["d"]
    token = 2 * H * (d / 2 + -(-d // 32))           # a token's codes and scales, keys and values
    if case["op"] != "attn":
        T = sum(rows)
        written = 2 * T * H * d * size[case["y"]]
        if case["op"] == "read":
            return {"bytes": T * token + written, "flops": 2 * T * H * d}
        return {"bytes": 2 * T * H * d * size[case["x"]] + 2 * T * token + written, "flops": 6 * T * H * d}
    read = pairs = 0
    for n, L in zip(rows, lens):
        w = case["window"] if case["causal"] and case["window"] else L
        read += min(L, n - 1 + w) if case["causal"] else L
        if not case["causal"]:
            pairs += n * L
        else:
            a = max(0, min(n, w - (L - n)))          # rows that see less than a whole window
            pairs += a * (L - n) + a * (a + 1) // 2 + (n - a) * w
    T = sum(rows)
    return {"bytes": read * token + T * case["heads"] * d * (size[case["q"]] + 2), "flops": 4 * pairs * case["heads"] * d}


# --------------------------------------------------------------------------- 64 bits

def _int8_64(case, seed):
    X, codes, sw = _int8_inputs(case, seed)
    w = codes.double() * sw.double()[:, None]
    out = torch.empty(case["T"], case["d_out"], dtype=torch.float64, device="cuda")
    for t0 in range(0, case["T"], 8192):
        x = X[t0:t0 + 8192].double()
        s = (x.abs().amax(dim=1, keepdim=True) / 127.0).float().double().clamp_min(2.0 ** -60)      # binary32, rounded once
        out[t0:t0 + 8192] = (torch.round((x / s).float().double()) * s) @ w.t()
    return out


def _mxfp4_64(x):
    """The values that MXFP4 holds of x [..., d], in 64 bits."""
    shape = x.shape
    x = torch.nn.functional.pad(x.double(), (0, -shape[-1] % 32))
    x = x.view(*shape[:-1], -1, 32)
    E = (torch.frexp(x.abs().amax(dim=-1, keepdim=True))[1] - 1 - 2).clamp_min(-127).double()
    y = x * torch.exp2(-E)
    a = y.abs()
    step = torch.where(a >= 4, 2.0, torch.where(a >= 2, 1.0, 0.5)).double()      # spacing of the grid at a
    v = (torch.round(a / step) * step).clamp_max(6.0) * torch.sign(y) * torch.exp2(E)
    return v.flatten(-2)[..., :shape[-1]]


def _attn64(case, seed):
    b, K, V, Q = _kv_inputs(case, seed)
    H, d = case["kv_heads"], case["d"]
    G = case["heads"] // H
    out = torch.empty(b["T"], case["heads"], d, dtype=torch.float64, device="cuda")
    t = k0 = 0
    for n, L in zip(b["rows"], b["lens"]):
        i, j = torch.arange(L - n, L, device="cuda")[:, None], torch.arange(L, device="cuda")[None]
        hide = None
        if case["causal"]:
            hide = j > i
            if case["window"]:
                hide |= i - j >= case["window"]
        for h in range(H):
            k, v = _mxfp4_64(K[k0:k0 + L, h]), _mxfp4_64(V[k0:k0 + L, h])
            for q0 in range(h * G, h * G + G):
                s = (Q[t:t + n, q0].to(torch.bfloat16).double() @ k.t()) / math.sqrt(d)
                if hide is not None:
                    s.masked_fill_(hide, -math.inf)
                out[t:t + n, q0] = torch.softmax(s, dim=1) @ v
        t += n
        k0 += L
    return out


def exact(case, seed):
    if case["op"] == "int8":
        return _int8_64(case, seed)
    if case["op"] == "attn":
        return _attn64(case, seed)
    _, K, V, _ = _kv_inputs(case, seed)
    out = [torch.empty(x.shape, dtype=torch.float64, device="cuda") for x in (K, V)]
    for o, x in zip(out, (K, V)):
        for t0 in range(0, len(x), 4096):
            o[t0:t0 + 4096] = _mxfp4_64(x[t0:t0 + 4096])
    return out
