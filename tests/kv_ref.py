"""Plain 64-bit forms of the INT8 layer, the 4-bit key/value cache and attention over it, from
their formulas in include/w4a4.h, and the error bounds the tests hold the kernels to."""
from __future__ import annotations

import math

import numpy as np
import torch

BF16_U = 2.0 ** -8       # half a unit in the last place of bf16, relative
F32_U = 2.0 ** -24

E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])


# --------------------------------------------------------------------------- INT8

def int8_quantize(x: np.ndarray):
    """Rows of binary32 values: codes int8, scales binary32; a row with a NaN or Inf has scale NaN and zero codes."""
    with np.errstate(all="ignore"):
        a = np.max(np.abs(x), axis=1)
        bad = ~np.isfinite(a)
        s = np.maximum(np.where(bad, np.float32(1), a) / np.float32(127), np.float32(2.0 ** -60)).astype(np.float32)
        q = np.rint((x / s[:, None]).astype(np.float32))
    q[bad] = 0
    s[bad] = np.nan
    return q.astype(np.int8), s


def int8_product(q, s, wq, ws):
    """(Y in 64 bits, bound on fl32(fl32(s_x s_w) fl32(sum))): three roundings."""
    y = (q.astype(np.float64) @ wq.astype(np.float64).T) * (s.astype(np.float64)[:, None] * ws.astype(np.float64)[None])
    return y, 3.01 * F32_U * np.abs(y)


# --------------------------------------------------------------------------- 4-bit codes

def mxfp4(x: np.ndarray):
    """x [..., d] binary32: nibbles uint8 [..., 32 G], scale codes uint8 [..., G], and the values
    they stand for, float64 [..., d]."""
    d = x.shape[-1]
    G = -(-d // 32)
    p = np.zeros(x.shape[:-1] + (32 * G,), np.float32)
    p[..., :d] = x
    p = p.reshape(x.shape[:-1] + (G, 32))
    with np.errstate(all="ignore"):
        amax = np.max(np.abs(p), axis=-1).astype(np.float32)
        bad = ~np.isfinite(amax)
        e = np.frexp(np.where(bad, 1, amax).astype(np.float64))[1] - 1 - 2          # floor(log2 amax) - 2
    e = np.where(amax == 0, -127, np.maximum(e, -127))
    y = np.where(bad[..., None], 0, p.astype(np.float64)) * 2.0 ** (-e.astype(np.float64))[..., None]
    a = np.abs(y)
    hi = np.clip(np.searchsorted(E2M1, a), 1, 7)
    lo = hi - 1
    dl, dh = a - E2M1[lo], E2M1[hi] - a
    code = np.where(dl < dh, lo, np.where(dl > dh, hi, np.where(lo % 2 == 0, lo, hi)))
    code = np.where(a >= 6, 7, code)
    nib = (code | np.where(bad[..., None], 0, np.signbit(p).astype(np.int64) << 3)).astype(np.uint8)
    sc = np.where(bad, 255, e + 127).astype(np.uint8)
    v = E2M1[code] * np.where(nib >= 8, -1.0, 1.0) * 2.0 ** e.astype(np.float64)[..., None]
    v = np.where(bad[..., None], np.nan, v)
    flat = x.shape[:-1] + (32 * G,)
    return nib.reshape(flat), sc, v.reshape(flat)[..., :d]


def d_pad(d: int) -> int:
    return -(-d // 32) * 32 if d <= 128 else -(-d // 64) * 64


def decode_block(raw: np.ndarray, d: int):
    """Nibbles [16, d_pad] and scale codes [16, d_pad / 32] of the keys and of the values in one
    block's bytes, from the layout's own description."""
    g = d_pad(d) // 32
    sg = g if g <= 2 else -(-g // 4) * 4
    assert raw.size == 512 * g + 32 * sg
    kn, vn = np.zeros((16, 32 * g), np.uint8), np.zeros((16, 32 * g), np.uint8)
    ks, vs = np.zeros((16, g), np.uint8), np.zeros((16, g), np.uint8)
    for t in range(16):
        for c in range(32 * g):
            dword = ((c // 8) % 4 * 16 + t) * g + c // 32
            kn[t, c] = raw[dword * 4 + c % 8 // 2] >> (4 * (c % 2)) & 15
            byte = (t // 4 * 16 + c % 16) * 4 * g + c // 32 * 4 + t % 4
            vn[t, c] = raw[256 * g + byte] >> (4 * (c % 32 // 16)) & 15
        for b in range(g):
            ks[t, b] = raw[512 * g + t * sg + b]
            vs[t, b] = raw[512 * g + 16 * sg + t // 4 * 4 * sg + b * 4 + t % 4]
    return kn, ks, vn, vs


# --------------------------------------------------------------------------- attention

def attention(q, k, v, scale, lo, hi, few):
    """One head of one sequence in 64 bits: q [n, d] (bf16 values), k, v [L, d] as cached; row i
    sees tokens lo[i] <= t < hi[i] (tokens that are not there are left out by the caller).  Returns
    (o, the bound of every output, and its square's expectation).

    The bound: a score is a sum of d exact products in binary32 (d + 8 roundings or truncations
    of 2^-23 of the sum of magnitudes, the scaling and the maximum's subtraction among them), which
    moves p by that much relatively (times 1.01 for the exponential's curvature and its own few
    ulps), in numerator and denominator; p is rounded to bf16 (to two terms where there are few rows);
    the sums over L tokens round 2 L + 16 times; the output rounds to bf16."""
    q, k, v = (torch.as_tensor(x, dtype=torch.float64) for x in (q, k, v))
    n, d = q.shape
    L = k.shape[0]
    t = torch.arange(L)[None]
    lo, hi = torch.as_tensor(lo)[:, None], torch.as_tensor(hi)[:, None]
    seen = (t >= lo) & (t < hi)
    s = torch.where(seen, (q @ k.t()) * scale, torch.full((n, L), -math.inf, dtype=torch.float64))
    mag = torch.where(seen, (q.abs() @ k.abs().t()) * scale, torch.zeros((), dtype=torch.float64))
    if L == 0:
        z = torch.zeros(n, d, dtype=torch.float64)
        return z, z, z
    m = s.amax(1, keepdim=True)
    p = torch.where(seen, torch.exp(s - torch.where(torch.isneginf(m), torch.zeros_like(m), m)), torch.zeros((), dtype=torch.float64))
    l = p.sum(1, keepdim=True)
    live = seen.any(1, keepdim=True) & ~(l == 0)
    nan_v = torch.isnan(v)
    vz = torch.where(nan_v, torch.zeros_like(v), v)
    ls = torch.where(live, l, torch.ones_like(l))
    o = (p @ vz) / ls
    o = torch.where((seen.double() @ nan_v.double()) > 0, torch.full_like(o, math.nan), o)
    o = torch.where(live, o, torch.zeros_like(o))
    a = (p @ vz.abs()) / ls
    delta = 1.01 * (d + 8) * 2.0 ** -23 * mag.amax(1, keepdim=True) + 2.0 ** -21
    up = BF16_U ** 2 if few else BF16_U
    tol = (2 * delta + up + (2 * L + 16) * 2.0 ** -23) * a
    # p below the smallest normal number, 2^-126, may be lost whole (exp and the matrix instructions
    # flush what lies below); the running maximum is at most 2^8 short, so that the largest p is at least
    # 2^-8 and the sum of L such losses moves o by at most L 2^-118 max |v|; so may an output below 2^-126
    tol = tol + L * 2.0 ** -118 * (vz.abs().amax() if L else 0.0) + 2.0 ** -126
    tol = tol + BF16_U * (o.abs() + tol)
    # independent roundings, each uniform within half a step at most: a third of their squares
    var = (BF16_U ** 2 / 3) * (o ** 2 + (0 if few else 1) * ((p ** 2) @ (vz ** 2)) / ls ** 2) + (2 * delta * a) ** 2
    return o, tol, var
