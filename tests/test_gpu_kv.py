"""The 4-bit key/value cache and attention over it on the GPU against their 64-bit forms: cached
bytes bit for bit, outputs within bounds derived from the roundings, at the sizes, masks and values where a path changes."""
import math

import numpy as np
import pytest
import torch

from bit_quantized_dit_amd import w4a4 as B
from tests import kv_ref as R

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


class Setup:
    """Sequences of `lens` tokens in shuffled pages of a cache that starts as 0xFF bytes (its scale
    codes are NaNs), all of them written."""

    def __init__(self, lens, H, D, page, dtype=BF16, seed=0, fill=True, spare=2, edit=None):
        print(f"kv lens={lens} H={H} D={D} page={page} {dtype}", flush=True)
        rng = np.random.default_rng(seed)
        self.lens, self.H, self.D, self.page = list(lens), H, D, page
        need = [-(-n // page) for n in lens]
        self.n_pages = sum(need) + spare
        order = rng.permutation(self.n_pages)
        self.table = np.full((len(lens), max(need + [1])), -1, np.int32)
        at = 0
        for i, n in enumerate(need):
            self.table[i, :n] = order[at:at + n]
            at += n
        n = sum(lens)
        self.K = (rng.standard_normal((n, H, D)) * np.where(rng.random(D) < 0.05, 6, 1)).astype(np.float32)
        self.V = (rng.standard_normal((n, H, D)) * 1.5).astype(np.float32)
        if dtype == BF16:
            self.K, self.V = (torch.from_numpy(x).bfloat16().float().numpy() for x in (self.K, self.V))
        if edit:
            edit(self)
        self.cache = B.kv_cache(self.n_pages, page, H, D)
        self.cache.data.fill_(255)
        self.pages = torch.from_numpy(self.table).cuda()
        self.start = np.concatenate([[0], np.cumsum(lens)])
        self.dtype = dtype
        if fill:
            self.append_all()

    def batch(self, rows, lens=None, max_rows=None, pages=None):
        start = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
        return B.kv_batch(torch.from_numpy(start).cuda(), torch.tensor(self.lens if lens is None else lens, dtype=torch.int32).cuda(),
                          self.pages if pages is None else pages, max_rows=max(list(rows) + [0]) if max_rows is None else max_rows)

    def dev(self, x):
        return torch.from_numpy(np.ascontiguousarray(x)).to(self.dtype).cuda()

    def append_all(self):
        B.w4a4_kv_append(self.dev(self.K), self.dev(self.V), self.batch(self.lens), self.cache)
        torch.cuda.synchronize()

    def values(self, i, heads=slice(None)):
        """Cached keys and values of sequence i, float64."""
        a, e = self.start[i], self.start[i + 1]
        return R.mxfp4(self.K[a:e, heads])[2], R.mxfp4(self.V[a:e, heads])[2]


def _guarded(shape, dtype, fill=7.0):
    n = int(np.prod(shape))
    buf = torch.full((n + 512,), fill, dtype=dtype, device="cuda")
    return buf, buf[256:256 + n].view(shape)


def _guards_hold(buf, fill=7.0):
    assert bool((buf[:256] == fill).all()) and bool((buf[-256:] == fill).all())


DIMS = [1, 31, 32, 33, 64, 72, 96, 100, 128, 130, 192, 200, 256]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("D", DIMS)
def test_append_and_read(D, dtype):
    s = Setup([37, 1, 0, 64, 18], 3, D, 16 if D % 2 else 48, dtype)
    raw = s.cache.data.cpu().numpy().reshape(s.n_pages, s.H, s.page // 16, -1)
    for i, n in enumerate(s.lens):
        kn, ks, _ = R.mxfp4(s.K[s.start[i]:s.start[i + 1]])
        vn, vs, _ = R.mxfp4(s.V[s.start[i]:s.start[i + 1]])
        G = ks.shape[-1]
        for q in range(-(-n // 16)):
            page, r = s.table[i, q * 16 // s.page], q % (s.page // 16)
            for h in range(s.H):
                got = R.decode_block(raw[page, h, r], D)
                m = min(16, n - 16 * q)
                sl = slice(16 * q, 16 * q + m)
                assert np.array_equal(got[0][:m, :32 * G], kn[sl, h]) and np.array_equal(got[1][:m, :G], ks[sl, h]), (i, q, h)
                assert np.array_equal(got[2][:m, :32 * G], vn[sl, h]) and np.array_equal(got[3][:m, :G], vs[sl, h]), (i, q, h)
                assert not got[0][:m, 32 * G:].any() and not got[2][:m, 32 * G:].any()
                for x in got:           # tokens past the last one: untouched
                    assert (x[m:] == (15 if x.shape[1] > R.d_pad(D) // 32 else 255)).all()
    for y in (F32, BF16):
        rows = [min(n, r) for n, r in zip(s.lens, [20, 1, 0, 64, 3])]
        kb, k = _guarded((sum(rows) + 5, s.H, D), y)
        vb, v = _guarded((sum(rows) + 5, s.H, D), y)
        B.w4a4_kv_read(s.batch(rows), s.cache, k, v)
        torch.cuda.synchronize()
        _guards_hold(kb), _guards_hold(vb)
        at = 0
        for i, r in enumerate(rows):
            wk, wv = s.values(i)
            assert np.array_equal(k[at:at + r].double().cpu().numpy(), wk[len(wk) - r:]), i
            assert np.array_equal(v[at:at + r].double().cpu().numpy(), wv[len(wv) - r:]), i
            at += r
        assert bool((k[at:] == 7).all()) and bool((v[at:] == 7).all())      # rows behind the last sequence


def test_special_values():
    """Zeros of both signs, subnormals, the largest numbers, ties of the grid, NaN and infinities,
    in one group each; the other groups keep their values."""
    def edit(s):
        for x in (s.K, s.V):
            x[0, 0] = 0
            x[1, 0, :32] = -0.0
            x[2, 0, :32] = 1e-42
            x[3, 0, :32] = 3.0e38
            x[4, 0, :16] = [6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, 7.9, -0.25, -0.75, -1.25, 0.2500001, 5.000001, 2.0 ** -20, -2.0 ** -140]
            x[5, 0, 40] = np.nan
            x[6, 0, 3] = np.inf
            x[7, 0, 90] = -np.inf
            x[8, 0, :32] = 2.0 ** -126
    s = Setup([40], 2, 96, 16, F32, edit=edit)
    k, v = (torch.empty(40, 2, 96, device="cuda") for _ in range(2))
    B.w4a4_kv_read(s.batch([40]), s.cache, k, v)
    wk, wv = s.values(0)
    for got, want in ((k, wk), (v, wv)):
        got = got.double().cpu().numpy()
        nan = np.isnan(want)
        assert nan.sum() == 3 * 32 and np.array_equal(np.isnan(got), nan)
        assert np.array_equal(got[~nan], want[~nan]) and np.array_equal(np.signbit(got[1]), np.signbit(want[1]))


def test_append_in_pieces():
    """Tokens one by one, and in runs that start and end inside a block, leave the same bytes as one call;
    so do inputs that are slices of one larger array."""
    s = Setup([70, 33], 5, 72, 32)
    whole = s.cache.data.clone()
    s.cache.data.fill_(255)
    at = [0, 0]
    for step in ([1, 5], [1, 1], [3, 0], [17, 16], [0, 11], [48, 0]):
        rows = [[s.start[i] + at[i], s.start[i] + at[i] + step[i]] for i in range(2)]
        at = [a + b for a, b in zip(at, step)]
        kv = np.concatenate([np.concatenate([s.K[a:b], s.V[a:b]], 1) for a, b in rows])
        fused = s.dev(np.concatenate([kv, kv[:, :1]], 1))           # [rows, 11, 72]
        B.w4a4_kv_append(fused[:, :5], fused[:, 5:10], s.batch(step, lens=at), s.cache)
    assert at == [70, 33]
    torch.cuda.synchronize()
    assert torch.equal(s.cache.data, whole)


def test_bad_positions_and_pages():
    """Positions below zero, pages that are not there, lengths and row numbers out of range."""
    s = Setup([40, 20], 2, 64, 16)
    before = s.cache.data.clone()
    bad = s.pages.clone()
    bad[0, 1], bad[1, 0] = s.n_pages, -5
    b = s.batch([44, 20], lens=[40, 20], pages=bad)        # four rows below position 0
    k, v = (torch.full((64, 2, 64), 7.0, device="cuda") for _ in range(2))
    B.w4a4_kv_read(b, s.cache, k, v)
    want = np.concatenate([np.zeros((4, 2, 64)), s.values(0)[0], s.values(1)[0]])
    want[4 + 16:4 + 32] = 0
    want[44:60] = 0
    assert np.array_equal(k.double().cpu().numpy(), want)
    B.w4a4_kv_append(torch.ones_like(k), torch.ones_like(v), b, s.cache)
    torch.cuda.synchronize()
    raw, old = (x.view(s.n_pages, -1) for x in (s.cache.data, before))
    changed = sorted(int(p) for p in range(s.n_pages) if not torch.equal(raw[p], old[p]))
    assert changed == sorted([int(s.table[0, 0]), int(s.table[0, 2]), int(s.table[1, 1])])
    # a table longer than the pool's, lens past the table, q_start past the rows, more rows than max_rows
    s = Setup([40], 2, 64, 16)
    q = torch.tensor([-3, 50], dtype=torch.int32, device="cuda")
    far = B.kv_batch(q, torch.tensor([1 << 30], dtype=torch.int32, device="cuda"), s.pages, max_rows=9)
    k = torch.full((40, 2, 64), 7.0, device="cuda")
    v = torch.full((40, 2, 64), 7.0, device="cuda")
    B.w4a4_kv_read(far, s.cache, k, v)                     # 48 positions, rows 0 .. 39 at 8 .. 47; 9 of them done
    assert np.array_equal(k[:9].double().cpu().numpy(), s.values(0)[0][8:17]) and bool((k[9:] == 7).all()) and bool((v[9:] == 7).all())


def _check_attention(s, rows, Hq, qt=BF16, causal=True, window=0, scale=None, lens=None, pages=None, there=None, q=None, max_rows=None, heads=None):
    """One call against the 64-bit form.  there(i, t): whether token t of sequence i has a page; heads: the
    key/value heads that are compared (all)."""
    lens = s.lens if lens is None else lens
    print(f"attention rows={rows} lens={lens} Hq={Hq} H={s.H} D={s.D} causal={causal} window={window} q={qt}", flush=True)
    rng = np.random.default_rng(5)
    n = sum(rows)
    if q is None:
        q = (rng.standard_normal((n, Hq, s.D)) * 2).astype(np.float32)
    _, Q = _guarded((n + 3, Hq, s.D), qt, float("nan"))
    Q[:n] = torch.from_numpy(q).to(qt)
    b = s.batch(rows, lens=lens, pages=pages, max_rows=max_rows)
    ws = torch.full((max(B.w4a4_kv_attention_workspace_size(n + 3, b, Hq, s.cache), 256) + 512,), 255, dtype=torch.uint8, device="cuda")
    buf, O = _guarded((n + 3, Hq, s.D), BF16)
    B.w4a4_kv_attention(Q, b, s.cache, O, ws[:-512], scale=scale, causal=causal, window=window)
    torch.cuda.synchronize()
    _guards_hold(buf)
    assert bool((ws[-512:] == 255).all()) and bool((O[n:] == 7).all())
    qb = torch.from_numpy(q).bfloat16().double()
    sc = s.D ** -0.5 if scale is None else scale
    # Where the header promises weights of two bf16 terms (d_pad up to 96: 64 stacked rows, above: 32), a weight is off by
    # 2^-16 of itself at most; elsewhere it is rounded to bf16 once, off by at most half a step, 2^-8 of itself, and
    # |sum dp v| / sum p <= 2^-8 sum p |v| / sum p, numerator and denominator being of the same p apart from that.
    few = (max(rows) if max_rows is None else max_rows) * (Hq // s.H) <= (64 if s.D <= 96 else 32)
    at, err2, var, nr2 = 0, 0.0, 0.0, 0.0
    for i, r in enumerate(rows):
        some = list(range(s.H)) if heads is None else heads
        k, v = s.values(i, some)
        k, v = k[:lens[i]], v[:lens[i]]
        pos = np.arange(lens[i] - r, lens[i])
        lo = np.maximum(pos - window + 1, 0) if causal and window else np.zeros(r, np.int64)
        hi = pos + 1 if causal else np.full(r, lens[i])
        if there is not None:
            keep = np.array([there(i, t) for t in range(lens[i])], bool)
            cum = np.concatenate([[0], np.cumsum(keep)])
            k, v = k[keep], v[keep]
            lo, hi = cum[np.clip(lo, 0, lens[i])], cum[np.clip(hi, 0, lens[i])]
        for h in [j * (Hq // s.H) + e for j in some for e in range(Hq // s.H)]:
            kh = some.index(h // (Hq // s.H))
            o, tol, va = R.attention(qb[at:at + r, h], k[:, kh], v[:, kh], sc, lo, hi, few)
            got = O[at:at + r, h].double().cpu()
            assert torch.equal(torch.isnan(got), torch.isnan(o)), f"sequence {i} head {h}: NaN pattern"
            ok = ~torch.isnan(o)
            d = (got - o).abs()
            if not bool((d <= tol)[ok].all()):
                j = int(torch.argmax(torch.where(ok, d - tol, torch.full_like(d, -1.0))))
                raise AssertionError(f"sequence {i} head {h}: row {j // s.D} channel {j % s.D}: off {float(d.flatten()[j]):.3e}, bound {float(tol.flatten()[j]):.3e}")
            err2 += float((d[ok] ** 2).sum())
            var += float(va[ok].sum())
            nr2 += float((o[ok] ** 2).sum())
        at += r
    # the sum of many independent roundings' squares: within a tenth where there are thousands
    assert err2 <= 1.21 * var + 1e-30 or n * len(some) * (Hq // s.H) * s.D < 4000, f"root mean square error {err2 ** 0.5:.3e}, bound {var ** 0.5:.3e}"
    return O[:n].clone()


FEW = [([1], [500], 4, 1), ([1, 1, 1], [1, 16, 33], 2, 2), ([1] * 5, [17, 31, 32, 0, 64], 8, 8), ([2, 1, 3], [40, 700, 3], 10, 2),
       ([4, 4], [130, 4], 12, 3), ([16], [90], 4, 2), ([9, 1], [2100, 60], 6, 1), ([1], [4096], 1, 1)]


@pytest.mark.parametrize("D", DIMS)
def test_attention_few_rows_widths(D):
    s = Setup([300, 45], 2, D, 16)
    _check_attention(s, [1, 1], 6)
    _check_attention(s, [7, 3], 6)
    _check_attention(s, [16, 11], 8, F32)


@pytest.mark.parametrize("causal,window", [(True, 0), (True, 40), (False, 0)])
@pytest.mark.parametrize("rows,lens,Hq,H", FEW)
def test_attention_few_rows(rows, lens, Hq, H, causal, window):
    s = Setup(lens, H, 128, 48)
    _check_attention(s, rows, Hq, BF16, causal, window)


MANY = [([70], [70], 2, 1), ([130, 65], [130, 65], 3, 3), ([200, 1, 90], [900, 1, 95], 4, 2), ([65], [2000], 1, 1), ([300], [333], 5, 1)]


@pytest.mark.parametrize("D", DIMS)
def test_attention_many_rows_widths(D):
    s = Setup([140, 75], 2, D, 32)
    _check_attention(s, [140, 70], 2)
    _check_attention(s, [33, 70], 4, F32)


@pytest.mark.parametrize("causal,window", [(True, 0), (True, 50), (False, 0)])
@pytest.mark.parametrize("rows,lens,Hq,H", MANY)
def test_attention_many_rows(rows, lens, Hq, H, causal, window):
    s = Setup(lens, H, 128, 16)
    _check_attention(s, rows, Hq, BF16, causal, window)


@pytest.mark.parametrize("D", [31, 64, 72, 128])
@pytest.mark.parametrize("causal,window", [(True, 0), (True, 70), (False, 0)])
def test_attention_of_many_heads(D, causal, window):
    """Enough heads that eight wavefronts share a tile: rows of one, part of one and several row tiles, pages that are
    not there, NaN keys and values."""
    def edit(s):
        s.V[150, 3, 0], s.K[160, 5, 1], s.V[3, 257, D - 1] = np.nan, np.inf, -np.inf
    s = Setup([333, 90], 260, D, 16, edit=edit)
    heads = [0, 3, 5, 130, 257, 259]
    _check_attention(s, [300, 90], 260, BF16, causal, window, heads=heads)
    _check_attention(s, [70, 1], 520, F32, causal, window, heads=heads)
    bad = s.pages.clone()
    bad[0, 4], bad[0, 20], bad[1, 5] = -1, s.n_pages, 1 << 30
    there = lambda i, t: not ((i == 0 and t // 16 in (4, 20)) or (i == 1 and t // 16 == 5))
    _check_attention(s, [300, 90], 260, BF16, causal, window, pages=bad, there=there, heads=heads)


@pytest.mark.parametrize("H,rows", [(300, 70), (3, 700)])
def test_attention_of_many_rows_in_ranges(H, rows):
    """Long sequences whose tokens are cut, for workgroups of eight and of four wavefronts."""
    s = Setup([1300], H, 64, 64)
    for causal in (True, False):
        _check_attention(s, [rows], H, causal=causal, heads=[0, 1, H - 1])
    s = Setup([5000, 900], 1, 64, 64)
    _check_attention(s, [80, 70], 1)


@pytest.mark.parametrize("rows", [[3, 2, 5], [90, 2, 70]])
def test_rows_that_see_nothing(rows):
    """Rows before the first token, sequences without tokens, windows over pages that are not there."""
    s = Setup([rows[0] - 2, 0, 200], 2, 64, 16)
    O = _check_attention(s, rows, 4)
    assert not bool(O[:2].any()) and not bool(O[rows[0]:rows[0] + 2].any())
    bad = s.pages.clone()
    bad[2, 3], bad[2, 12] = -1, s.n_pages
    there = lambda i, t: not (i == 2 and t // 16 in (3, 12))
    _check_attention(s, rows, 4, pages=bad, there=there)
    _check_attention(s, rows, 4, pages=bad, there=there, causal=False)
    O = _check_attention(s, rows, 4, pages=bad, there=there, window=3)
    bad[2] = -1
    O = _check_attention(s, rows, 4, pages=bad, there=lambda i, t: i != 2)
    assert not bool(O[sum(rows[:2]):].any())


@pytest.mark.parametrize("rows", [[6], [100]])
def test_nan_in_and_out_of_sight(rows):
    """A NaN key makes the rows that see it NaN; a NaN value its 32 channels; rows that do not see
    them are as without them, and so is what lies behind the last token."""
    n, r = 230, rows[0]
    clean = Setup([n], 2, 96, 16)
    want = _check_attention(clean, rows, 4)

    def key(s): s.K[n - 3, 0, 5] = np.nan
    O = _check_attention(Setup([n], 2, 96, 16, edit=key), rows, 4)
    seen = torch.zeros(r, 4, 96, dtype=torch.bool, device="cuda")
    seen[r - 3:, :2] = True
    assert torch.equal(torch.isnan(O), seen) and torch.equal(O[~seen], want[~seen])

    def value(s): s.V[n - 3, 1, 70] = np.inf
    O = _check_attention(Setup([n], 2, 96, 16, edit=value), rows, 4)
    seen.zero_()
    seen[r - 3:, 2:, 64:] = True
    assert torch.equal(torch.isnan(O), seen) and torch.equal(O[~seen], want[~seen])

    def early(s): s.V[4, 0, 0], s.K[9, 1, 95] = np.nan, -np.inf
    O = _check_attention(Setup([n], 2, 96, 16, edit=early), rows, 4)
    assert bool(torch.isnan(O[:, :2, :32]).all()) and not bool(torch.isnan(O[:, :2, 32:]).any()) and bool(torch.isnan(O[:, 2:]).all())
    windowed = _check_attention(clean, rows, 4, window=20)
    assert torch.equal(_check_attention(Setup([n], 2, 96, 16, edit=early), rows, 4, window=20), windowed)
    O = _check_attention(Setup([n], 2, 96, 16, edit=lambda s: s.V.__setitem__((n - r, 0, 0), np.nan)), rows, 4, causal=False)
    assert bool(torch.isnan(O[:, :2, :32]).all()) and not bool(torch.isnan(O[:, 2:]).any())


@pytest.mark.parametrize("rows", [[1], [80]])
def test_large_scores(rows):
    """Scores far apart, equal, and past the range of exp; infinite queries make their own row NaN."""
    s = Setup([400], 1, 64, 64)
    rng = np.random.default_rng(3)
    q = (rng.standard_normal((rows[0], 2, 64)) * 300).astype(np.float32)
    _check_attention(s, rows, 2, q=q)
    _check_attention(s, rows, 2, q=np.zeros_like(q))
    _check_attention(s, rows, 2, scale=1e-6)
    q = (rng.standard_normal((rows[0], 2, 64))).astype(np.float32)
    q[0, 1, 3] = np.inf
    n = rows[0]
    O = torch.empty(n, 2, 64, dtype=BF16, device="cuda")
    b = s.batch(rows)
    B.w4a4_kv_attention(torch.from_numpy(q).cuda(), b, s.cache, O, B.alloc_workspace_kv(n, b, 2, s.cache))
    assert bool(torch.isnan(O[0, 1]).all()) and int(torch.isnan(O).sum()) == 64


def test_long_ranges_are_joined():
    """Lengths that are cut into ranges, with a table that holds far more than the sequences do."""
    s = Setup([5000, 300, 1], 2, 64, 16)
    wide = torch.full((3, 4000), -1, dtype=torch.int32, device="cuda")
    wide[:, :s.pages.shape[1]] = s.pages
    a = _check_attention(s, [1, 1, 1], 4, pages=wide)
    _check_attention(s, [3, 1, 1], 4, pages=wide, causal=False)
    _check_attention(s, [100, 80, 1], 2, pages=wide)
    b = _check_attention(s, [1, 1, 1], 4, pages=wide)
    assert torch.equal(a, b)


@pytest.mark.parametrize("window", [500, 530, 1000, 1023, 1025, 2500, 1 << 40])
def test_windows_that_are_cut(window):
    """Windows of several ranges that start and end inside a step."""
    s = Setup([3001, 1040, 700], 2, 32, 16)
    for rows in ([1, 1, 1], [7, 2, 3], [9, 16, 1]):
        _check_attention(s, rows, 2, window=window)
    _check_attention(s, [100, 70, 1], 2, window=window)


@pytest.mark.parametrize("n", [64, 65, 70])
def test_many_rows_of_many_sequences(n):
    """Row tiles counted by a wavefront's lanes, and of more sequences; some without rows."""
    lens = [37 * i % 211 for i in range(n)]
    rows = [0 if i % 5 == 4 else min(lens[i], 13 * i % 80) for i in range(n)]
    rows[3] = lens[3] = 150
    s = Setup(lens, 1, 32, 16)
    _check_attention(s, rows, 1)
    _check_attention(s, rows, 2, window=40)


@pytest.mark.parametrize("n,H,Hq", [(65, 1, 1), (130, 2, 10), (300, 1, 4), (1100, 1, 2)])
def test_many_sequences(n, H, Hq):
    """More sequences than a wavefront has lanes, some without rows or tokens, a few long, in a table of long ones."""
    rng = np.random.default_rng(n)
    lens = [int(x) for x in rng.choice([0, 1, 15, 40, 200], n)]
    lens[3], lens[n - 2] = 1500, 2100
    rows = [int(x) for x in rng.choice([0, 1, 1, 2], n)]
    rows[3], rows[n - 2], rows[n - 1] = 1, 2, 1
    s = Setup(lens, H, 32, 16)
    wide = torch.full((n, 2000), -1, dtype=torch.int32, device="cuda")
    wide[:, :s.pages.shape[1]] = s.pages
    _check_attention(s, rows, Hq, pages=wide)


def test_cache_past_four_gigabytes():
    """Blocks whose offsets need more than 32 bits, and those in front of them left alone."""
    H, D, page = 8, 128, 64
    page_bytes = H * page // 16 * 2176
    n_pages = (5 << 30) // page_bytes
    cache = B.kv_cache(n_pages, page, H, D)
    assert cache.data.numel() > 1 << 32
    g = torch.Generator(device="cuda").manual_seed(2)
    K, V = (torch.randn(200, H, D, device="cuda", generator=g).bfloat16() for _ in range(2))
    pages = torch.tensor([[n_pages - 1, 0, n_pages - 3, n_pages // 2]], dtype=torch.int32, device="cuda")
    used = sorted(pages[0].tolist())
    for p in used:
        cache.data[p * page_bytes:(p + 1) * page_bytes].fill_(255)
    marks = [p * page_bytes - 16 for p in used if p] + [(p + 1) * page_bytes for p in used if p + 1 < n_pages]
    for m in marks:
        cache.data[m:m + 16] = 77
    lens = torch.tensor([200], dtype=torch.int32, device="cuda")
    b = B.kv_batch(torch.tensor([0, 200], dtype=torch.int32, device="cuda"), lens, pages, max_rows=200)
    B.w4a4_kv_append(K, V, b, cache)
    k, v = torch.empty_like(K), torch.empty_like(V)
    B.w4a4_kv_read(b, cache, k, v)
    for got, x in ((k, K), (v, V)):
        assert np.array_equal(got.double().cpu().numpy(), R.mxfp4(x.float().cpu().numpy())[2])
    assert all(bool((cache.data[m:m + 16] == 77).all()) for m in marks)
    for n in (1, 80):
        Q = torch.randn(n, H, D, device="cuda", generator=g).bfloat16()
        O = torch.empty_like(Q)
        bq = B.kv_batch(torch.tensor([0, n], dtype=torch.int32, device="cuda"), lens, pages, max_rows=n)
        B.w4a4_kv_attention(Q, bq, cache, O, B.alloc_workspace_kv(n, bq, H, cache), causal=False)
        kd, vd = k.double().cpu(), v.double().cpu()
        for h in range(H):
            o, tol, _ = R.attention(Q[:, h].double().cpu(), kd[:, h], vd[:, h], D ** -0.5, np.zeros(n, int), np.full(n, 200), n <= 64)
            assert bool(((O[:, h].double().cpu() - o).abs() <= tol).all())


def test_more_rows_than_max_rows():
    s = Setup([200], 1, 64, 16)
    q = np.random.default_rng(1).standard_normal((150, 2, 64)).astype(np.float32)
    full = _check_attention(s, [150], 2, q=q)
    for most in (4, 100):
        O = torch.full((150, 2, 64), 7.0, dtype=BF16, device="cuda")
        b = s.batch([150], max_rows=most)
        B.w4a4_kv_attention(torch.from_numpy(q).cuda().bfloat16(), b, s.cache, O, B.alloc_workspace_kv(150, b, 2, s.cache))
        assert bool((O[most:] == 7).all())
        assert float((O[:most].float() - full[:most].float()).abs().max()) <= 0.03      # another kernel: both within a few roundings of values of 1.5


def test_strided_queries_and_streams():
    """Q as a slice of a fused projection, on a stream of the caller's own."""
    s = Setup([300, 120], 2, 72, 16)
    for rows in ([1, 1], [100, 70]):
        n = sum(rows)
        fused = torch.randn(n, 6 + 4, 72, device="cuda").bfloat16()
        b = s.batch(rows)
        ws = B.alloc_workspace_kv(n, b, 6, s.cache)
        want = torch.empty(n, 6, 72, dtype=BF16, device="cuda")
        B.w4a4_kv_attention(fused[:, :6].contiguous(), b, s.cache, want, ws)
        torch.cuda.synchronize()
        st = torch.cuda.Stream()
        got = torch.empty_like(want)
        st.wait_stream(torch.cuda.current_stream())
        B.w4a4_kv_attention(fused[:, :6], b, s.cache, got, ws, stream=st)
        st.synchronize()
        assert torch.equal(got, want)


def test_decoding_loop_in_a_graph():
    """Append, then attend, captured once and replayed while lens, pages and inputs change; every
    replay equals eager calls on a second cache.  Two graphs share the workspace."""
    H, Hq, D, page = 2, 8, 64, 16
    start = [29, 500, 0]
    pages = torch.arange(3 * 40, dtype=torch.int32, device="cuda").view(3, 40)
    caches = [B.kv_cache(120, page, H, D) for _ in range(2)]
    q_start = torch.arange(4, dtype=torch.int32, device="cuda")
    lens = torch.tensor(start, dtype=torch.int32, device="cuda")
    K, V = (torch.randn(3, H, D, device="cuda").bfloat16() for _ in range(2))
    Q = torch.randn(3, Hq, D, device="cuda").bfloat16()
    b = B.kv_batch(q_start, lens, pages, max_rows=1)
    old = [torch.randn(sum(start), H, D, device="cuda").bfloat16() for _ in range(2)]
    fill = B.kv_batch(torch.tensor([0, 29, 529, 529], dtype=torch.int32, device="cuda"), lens.clone(), pages, max_rows=500)
    for c in caches:
        B.w4a4_kv_append(*old, fill, c)
    ws = B.alloc_workspace_kv(3, b, Hq, caches[0])
    O = [torch.empty(3, Hq, D, dtype=BF16, device="cuda") for _ in range(3)]

    def step(c, o, causal=True):
        B.w4a4_kv_append(K, V, b, c)
        B.w4a4_kv_attention(Q, b, c, o, ws, causal=causal)
    lens += 1
    step(caches[0], O[0])
    torch.cuda.synchronize()
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for g, o, causal in zip(graphs, O, (True, False)):
        with torch.cuda.graph(g):
            step(caches[0], o, causal)
    for i in range(6):
        for t in (K, V, Q):
            t.normal_()
        for g in graphs:
            g.replay()
        step(caches[1], O[2])
        torch.cuda.synchronize()
        assert torch.equal(O[0], O[2]) and torch.equal(O[1], O[2]), i      # one row a sequence: causal sees every token
        lens += 1


def test_refusals():
    s = Setup([20], 2, 64, 16)
    b = s.batch([1])
    Q, O = torch.zeros(1, 4, 64, device="cuda"), torch.zeros(1, 4, 64, dtype=BF16, device="cuda")
    ws = B.alloc_workspace_kv(1, b, 4, s.cache)
    for bad in (dict(scale=0.0), dict(scale=float("nan")), dict(window=-1), dict(causal=False, window=3)):
        with pytest.raises(B.W4A4Error):
            B.w4a4_kv_attention(Q, b, s.cache, O, ws, **bad)
    with pytest.raises(B.W4A4Error):
        B.w4a4_kv_attention(Q[:, :3], b, s.cache, O[:, :3].contiguous(), ws)
    with pytest.raises(TypeError):
        B.w4a4_kv_attention(Q.half(), b, s.cache, O, ws)
    with pytest.raises(TypeError):
        B.w4a4_kv_attention(Q, b, s.cache, O.float(), ws)
    with pytest.raises(ValueError):
        B.w4a4_kv_attention(Q[:, :, :32], b, s.cache, O, ws)
    with pytest.raises(ValueError):
        B.w4a4_kv_attention(Q, b, s.cache, O[:, ::2], ws)
    K = torch.zeros(1, 2, 64, device="cuda")
    with pytest.raises(ValueError):
        B.w4a4_kv_append(K, K.bfloat16(), b, s.cache)
    with pytest.raises(ValueError):
        B.w4a4_kv_append(K.transpose(1, 2).contiguous().transpose(1, 2), K, b, s.cache)
    with pytest.raises(ValueError):
        B.w4a4_kv_append(K.cpu(), K.cpu(), b, s.cache)
    with pytest.raises(TypeError):
        B.kv_batch(b.keep[0].long(), b.keep[1], b.keep[2], max_rows=1)
    with pytest.raises(ValueError):
        B.kv_batch(b.keep[0], b.keep[1], b.keep[2][:, :0], max_rows=1)
    B.w4a4_kv_append(K[:0], K[:0], s.batch([0]), s.cache)
