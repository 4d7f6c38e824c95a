"""Plain 64-bit forms of the FP8 block-scaled layer and the mixture-of-experts layer, from
their formulas in include/w4a4.h, and the error bounds the tests hold the kernels to."""
from __future__ import annotations

import numpy as np

# E4M3 values by code (0x7F and 0xFF are NaN)
_c = np.arange(256)
_e, _m = (_c >> 3) & 15, _c & 7
VALUE = np.where(_e == 0, _m * 2.0 ** -9, (1 + _m / 8) * 2.0 ** (_e - 7.0)) * np.where(_c >= 128, -1.0, 1.0)
VALUE[[0x7F, 0xFF]] = np.nan
_GRID = VALUE[:0x7F]                                     # 0 .. 448, ascending


def encode(q: np.ndarray) -> np.ndarray:
    """Codes nearest to q (|q| <= 448 up to rounding), ties to the even code, sign kept."""
    a = np.abs(q.astype(np.float64))
    hi = np.clip(np.searchsorted(_GRID, a), 1, len(_GRID) - 1)
    lo = hi - 1
    dl, dh = a - _GRID[lo], _GRID[hi] - a
    code = np.where(dl < dh, lo, np.where(dl > dh, hi, np.where(lo % 2 == 0, lo, hi)))
    return (code | (np.signbit(q).astype(np.int64) << 7)).astype(np.uint8)


def scale_of(amax: np.ndarray, kind: int) -> np.ndarray:
    """Scales (binary32) of blocks with largest magnitude amax (binary32)."""
    amax = amax.astype(np.float32)
    bad = ~np.isfinite(amax)
    a = np.where(bad, np.float32(1), amax)
    if kind == 0:
        s = np.maximum(a / np.float32(448), np.float32(2.0 ** -60))
    else:
        e = np.ceil(np.log2(np.maximum(a.astype(np.float64), 2.0 ** -140) / 448.0))
        e = np.where(a > 448.0 * 2.0 ** e, e + 1, np.where(a <= 448.0 * 2.0 ** (e - 1), e - 1, e))
        s = 2.0 ** np.maximum(e, -60.0)
    return np.where(bad, np.float32(np.nan), s.astype(np.float32))


def _codes(x: np.ndarray, s: np.ndarray) -> np.ndarray:
    """x and its scales, broadcast, to codes; blocks with a NaN scale are zero."""
    bad = np.isnan(s)
    with np.errstate(all="ignore"):
        q = (x.astype(np.float32) / np.where(bad, np.float32(1), s)).astype(np.float32)
    return np.where(np.broadcast_to(bad, q.shape), 0, encode(np.where(np.broadcast_to(bad, q.shape), 0, q))).astype(np.uint8)


def quantize_rows(x: np.ndarray, kind: int):
    """Activations [T, d] (binary32): codes [T, k_pad], scales [T, k_pad / 128]."""
    T, d = x.shape
    kb = -(-d // 128)
    p = np.zeros((T, kb * 128), np.float32)
    p[:, :d] = x
    p = p.reshape(T, kb, 128)
    with np.errstate(invalid="ignore"):
        s = scale_of(np.max(np.abs(p), axis=2), kind)
    return _codes(p, s[:, :, None]).reshape(T, kb * 128), s


def quantize_blocks(w: np.ndarray, kind: int):
    """Weights [rows, cols] (binary32): codes [rows, cols], scales [rows/128, cols/128] (rounded up)."""
    r, c = w.shape
    rb, cb = -(-r // 128), -(-c // 128)
    p = np.zeros((rb * 128, cb * 128), np.float32)
    p[:r, :c] = w
    b = p.reshape(rb, 128, cb, 128)
    with np.errstate(invalid="ignore"):
        s = scale_of(np.max(np.abs(b), axis=(1, 3)), kind)
    return _codes(b, s[:, None, :, None]).reshape(rb * 128, cb * 128)[:r, :c].copy(), s


def dequant_rows(codes, s):
    return VALUE[codes] * np.repeat(s.astype(np.float64), 128, axis=1)


def dequant_blocks(codes, s):
    r, c = codes.shape
    return VALUE[codes] * np.repeat(np.repeat(s.astype(np.float64), 128, 0)[:r], 128, 1)[:, :c]


# Products of the FP8 matrix instructions (many tokens, bf16 outputs) lose what is 13 bits below
# the largest product beside them: at most 2^-12.5 of a block's largest product was seen per
# block of 128, and that is at most this share of the sum of magnitudes.
FP8_MFMA = 2.0 ** -12


def product(xd: np.ndarray, wd: np.ndarray, fp8_mfma: bool = False):
    """(X W^T, bound on a binary32 evaluation of it): within a block at most 128 additions of
    exact products, then one scaling, one addition per block and at most 16 joins of partial
    sums; each rounds by at most 2^-23 of the sum of magnitudes (2^-24, doubled for a matrix
    unit that truncates).  fp8_mfma adds what the FP8 matrix instructions drop."""
    with np.errstate(all="ignore"):
        y = xd @ wd.T
        mag = np.abs(xd) @ np.abs(wd).T
    nkb = -(-xd.shape[1] // 128)
    return y, ((128 + 2 + nkb + 16) * 2.0 ** -23 + (FP8_MFMA if fp8_mfma else 0.0)) * mag


BF16_U = 2.0 ** -8      # half a unit in the last place of bf16, relative


def bf16(x: np.ndarray) -> np.ndarray:
    """Nearest-even bf16 of binary32 values, as binary32 (finite values)."""
    u = x.astype(np.float32).view(np.uint32).astype(np.uint64)
    return ((u + 0x7FFF + ((u >> 16) & 1)) & 0xFFFF0000).astype(np.uint32).view(np.float32)


def topk(logits: np.ndarray, k: int) -> np.ndarray:
    """Indices of the k largest, larger first, ties to the lower index, NaN first."""
    out = np.empty((logits.shape[0], k), np.int64)
    for t, l in enumerate(logits):
        order = sorted(range(len(l)), key=lambda e: (0, 0.0, e) if np.isnan(l[e]) else (1, -float(l[e]), e))
        out[t] = order[:k]
    return out


def close(got, want, tol, what):
    got, want = np.asarray(got, np.float64), np.asarray(want, np.float64)
    assert got.shape == want.shape, what
    nan = np.isnan(want)
    assert np.array_equal(np.isnan(got), nan), f"{what}: NaN pattern differs"
    d = np.abs(got - want)[~nan]
    t = np.broadcast_to(tol, want.shape)[~nan]
    bad = d > t
    if bad.any():
        i = int(np.argmax(d - t))
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} outside the bound; worst off {d[i]:.3e}, bound {t[i]:.3e}")
